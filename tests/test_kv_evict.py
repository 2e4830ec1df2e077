"""attn_kv_select_paged and attn_kv_compact_paged: refusals on the CPU; on the GPU the choice against a sort on the host and
every byte of the caches against a copy row by row; then a decode that accumulates, evicts and goes on."""
import math

import numpy as np
import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def A():
    ensure_built()
    import exact_softmax_attention_gb300 as mod
    return mod


# ------------------------------------------------------------------------------------- CPU

def select_status(A, **kw):
    a = dict(score=0x1000, page_table=0x2000, seqlens=0x3000, kept=0x4000, new_seqlens=0x5000, page_size=16, B=0, Hkv=2, max_pages_per_seq=4,
             num_pages=8, budget=10, sinks=2, recent=3)
    a.update(kw)
    return A.attn_kv_select_paged(**a, stream=0, raise_on_error=False)


def compact_status(A, **kw):
    a = dict(k_cache=0x1000, v_cache=0x2000, score=0x3000, kept=0x4000, new_seqlens=0x5000, page_table=0x6000, page_size=16, B=0, Hkv=2, d=64,
             max_pages_per_seq=4, num_pages=8, budget=10, kv_format="bf16")
    a.update(kw)
    return A.attn_kv_compact_paged(**a, stream=0, raise_on_error=False)


def test_refusals(A):
    null, shape, align, arg = A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    sizes = (dict(B=-1), dict(B=65536), dict(Hkv=0), dict(Hkv=65536), dict(page_size=0), dict(max_pages_per_seq=0), dict(num_pages=0),
             dict(num_pages=1 << 27), dict(max_pages_per_seq=1 << 26), dict(budget=0), dict(budget=-4), dict(B=65535, Hkv=65535))
    for f, names in ((select_status, ("score", "page_table", "seqlens", "kept", "new_seqlens")),
                     (compact_status, ("k_cache", "v_cache", "kept", "new_seqlens", "page_table"))):
        assert f(A) == A.ATTN_OK
        for name in names:
            assert f(A, **{name: None}) == null, name
            assert f(A, **{name: 0x7002}) == align, name
        for bad in sizes:
            assert f(A, **bad) == shape, bad
    for bad in (dict(sinks=-1), dict(recent=-1), dict(sinks=8), dict(recent=9), dict(sinks=2**31 - 1, recent=2**31 - 1)):
        assert select_status(A, **bad) == shape, bad
    assert select_status(A, sinks=7) == A.ATTN_OK and select_status(A, sinks=0, recent=10) == A.ATTN_OK
    assert select_status(A, new_seqlens=0x3000) == arg
    assert compact_status(A, score=None) == A.ATTN_OK and compact_status(A, score=0x3002) == align
    for bad in (dict(d=0), dict(d=24), dict(d=272), dict(d=-16)):
        assert compact_status(A, **bad) == shape, bad
    for bad in (3, -1):
        assert compact_status(A, kv_format=bad) == arg
    for bad in (dict(k_cache=0x1008), dict(v_cache=0x2004)):
        assert compact_status(A, **bad) == align


def wanted(score, len_, budget, sinks, recent):
    """kept row of one sequence and head from the scores of its tokens (float32), by a stable sort."""
    kept = np.full(budget, -1, np.int32)
    if len_ <= budget:
        kept[:len_] = np.arange(len_)
        return kept
    end, stop = budget - recent, len_ - recent
    key = np.where(np.isnan(score), np.inf, score.astype(np.float64) + 0.0)
    middle = sorted(range(sinks, stop), key=lambda i: (not np.isnan(score[i]), -key[i], i))[:end - sinks]
    stays = set(middle)
    behind = iter(sorted(i for i in middle if i >= end))
    kept[:sinks] = np.arange(sinks)
    kept[sinks:end] = [j if j in stays else next(behind) for j in range(sinks, end)]
    kept[end:] = np.arange(stop, len_)
    return kept


def test_the_oracle_itself():
    """Known answers, and what the documentation promises of every choice."""
    s = np.array([0, 5, 1, 5, 0, 9, 2, 5, 3, 0], np.float32)
    assert wanted(s, 10, 4, 0, 0).tolist() == [5, 1, 7, 3]
    assert wanted(s, 10, 4, 1, 1).tolist() == [0, 1, 5, 9]
    assert wanted(s, 10, 4, 4, 0).tolist() == [0, 1, 2, 3] and wanted(s, 10, 4, 0, 4).tolist() == [6, 7, 8, 9]
    assert wanted(s, 3, 4, 1, 1).tolist() == [0, 1, 2, -1]
    s = np.array([np.nan, -np.inf, np.inf, -0.0, 0.0, -1], np.float32)
    assert wanted(s, 6, 2, 0, 0).tolist() == [0, 2] and wanted(s, 6, 3, 0, 0).tolist() == [0, 3, 2]
    rs = np.random.RandomState(0)
    for _ in range(200):
        n, k = rs.randint(1, 60), rs.randint(1, 40)
        sinks = rs.randint(0, k + 1)
        recent = rs.randint(0, k - sinks + 1)
        kept = wanted(rs.randint(0, 4, n).astype(np.float32), n, k, sinks, recent)
        new = min(n, k)
        assert (kept[:new] >= np.arange(new)).all() and len(set(kept[:new])) == new and (kept[new:] == -1).all()


# ------------------------------------------------------------------------------------- GPU

class Cache:
    def __init__(self, lens, Hkv, d, page, fmt="bf16", seed=0, values="sums"):
        rs = np.random.RandomState(seed + d + page + len(lens))
        self.lens, self.B, self.Hkv, self.d, self.page, self.fmt = np.array(lens), len(lens), Hkv, d, page, fmt
        pages = -(-self.lens // page)
        self.num, self.width = int(pages.sum()) + 2, int(max(1, pages.max())) + 1
        perm, self.pt, at = rs.permutation(self.num), np.full((self.B, self.width), 2**31 - 1, np.int32), 0
        for b, c in enumerate(pages):
            self.pt[b, :c] = perm[at:at + c]
            at += c
        shape = (self.num, Hkv, page)
        if values == "sums":
            score = np.where(rs.rand(*shape) < 0.2, 0.0, np.exp(2 * rs.standard_normal(shape)))
        elif values == "few":
            score = rs.randint(0, 3, shape)
        elif values == "equal":
            score = np.full(shape, 2.5)
        else:  # every kind of number
            pool = np.array([np.nan, np.inf, -np.inf, -0.0, 0.0, 1.0, -1.0, 1e-45, -1e-45, 3e38, -3e38, 1.0000001], np.float32)
            score = pool[rs.randint(0, len(pool), shape)]
        self.score = torch.from_numpy(score.astype(np.float32)).to(DEV)
        t = torch.int16 if fmt == "bf16" else torch.uint8
        self.kc, self.vc = (torch.from_numpy(rs.randint(0, 2**15 if fmt == "bf16" else 256, (self.num, page, Hkv, d))).to(DEV).to(t) for _ in range(2))
        self.ptd, self.lend = torch.from_numpy(self.pt).to(DEV), torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        self.new = torch.full((self.B,), -7, dtype=torch.int32, device=DEV)

    def select(self, A, budget, sinks, recent):
        self.budget = budget
        self.kept = torch.full((self.B, self.Hkv, budget), -9, dtype=torch.int32, device=DEV)
        A.attn_kv_select_paged(self.score, self.ptd, self.lend, self.kept, self.new, self.page, self.B, self.Hkv, self.width, self.num, budget, sinks,
                               recent)

    def compact(self, A, score=True):
        A.attn_kv_compact_paged(self.kc, self.vc, self.score if score else None, self.kept, self.new, self.ptd, self.page, self.B, self.Hkv, self.d,
                                self.width, self.num, self.budget, self.fmt)

    def place(self, b, tok):
        tok = np.asarray(tok)
        return self.pt[b, tok // self.page].astype(np.int64), tok % self.page

    def expect(self, kept):
        """(k, v, score) after moving the rows of kept (host), from copies"""
        out = [x.cpu().numpy() for x in (self.kc, self.vc, self.score)]
        old = [x.copy() for x in out]
        for b in range(self.B):
            for h in range(self.Hkv):
                j = np.flatnonzero(kept[b, h] >= 0)
                (dp, ds), (sp, ss) = self.place(b, j), self.place(b, kept[b, h, j])
                for x, o in zip(out[:2], old):
                    x[dp, ds, h] = o[sp, ss, h]
                out[2][dp, h, ds] = old[2][sp, h, ss]
        return out


CASES = [  # lengths, Hkv, page, budget, sinks, recent
    ([1], 1, 1, 1, 0, 0),
    ([2], 1, 16, 1, 0, 0),
    ([10, 0, 1, 300, 64, 65], 2, 16, 64, 4, 8),
    ([40, 33, 32, 31], 3, 7, 32, 0, 32),       # only the last ones stay
    ([40, 33], 1, 5, 32, 32, 0),               # only the first ones
    ([40, 33], 1, 5, 32, 0, 0),
    ([1000, 1024, 1025, 2048, 2049], 2, 16, 1000, 4, 100),
    ([3000, 700], 2, 256, 2990, 4, 2000),      # a few leave, the last ones shift by less than their number
    ([16384 + 37, 16384 + 36], 1, 64, 20, 4, 16),
    ([16400], 2, 16, 16399, 10, 6),
    ([16390, 40000], 1, 16, 9000, 0, 20),      # keys not held in registers, holes in several turns
    ([30000], 1, 1, 14000, 1, 0),
    ([14000], 1, 16, 12000, 0, 0),             # held, holes in one turn
    ([16000], 2, 16, 8000, 0, 0),
    ([33000, 20000, 900], 1, 16, 15000, 6, 5000),  # several blocks for each row, the slots' end within one of them
    ([70000], 3, 12, 512, 2, 64),
    ([400000, 5], 1, 64, 3000, 4, 10),             # more than their shared memories hold
    ([390000], 1, 16, 380000, 0, 7),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hkv,page,budget,sinks,recent", CASES)
@pytest.mark.parametrize("values", ["sums", "few", "equal", "all"])
def test_select_and_compact(A, lens, Hkv, page, budget, sinks, recent, values):
    c = Cache(lens, Hkv, 16, page, values=values)
    c.select(A, budget, sinks, recent)
    assert A.attn_get_device_status() == 0
    score = c.score.cpu().numpy()
    want = np.stack([[wanted(score[c.place(b, np.arange(n))[0], h, c.place(b, np.arange(n))[1]], int(n), budget, sinks, recent)
                      for h in range(Hkv)] for b, n in enumerate(c.lens)])
    assert np.array_equal(c.kept.cpu().numpy(), want)
    assert np.array_equal(c.new.cpu().numpy(), np.minimum(c.lens, budget))
    expect = c.expect(want)
    c.compact(A)
    assert A.attn_get_device_status() == 0
    for got, ref in zip((c.kc, c.vc, c.score), expect):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=got.dtype == torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("d", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("lens,Hkv,budget", [([900], 1, 500), ([70, 300, 20], 3, 60), ([200] * 90, 5, 150)])
@pytest.mark.parametrize("score", [True, False])
def test_compact_rows(A, fmt, d, lens, Hkv, budget, score):
    """Rows of every width, few and many blocks, with and without scores; any choice with kept[j] >= j."""
    c = Cache(lens, Hkv, d, 7, fmt, seed=1)
    rs = np.random.RandomState(2)
    kept = np.full((c.B, Hkv, budget), -1, np.int32)
    new = np.minimum(c.lens, budget)
    for b in range(c.B):
        for h in range(Hkv):
            if rs.rand() < 0.5:
                kept[b, h, :new[b]] = np.sort(rs.permutation(c.lens[b])[:new[b]])  # ascending
            else:
                kept[b, h, :new[b]] = [rs.randint(j, c.lens[b]) for j in range(new[b])]  # repeated ones among them
    kept[0, 0, 3] = -1  # no token: the slot stays
    c.kept, c.budget = torch.from_numpy(kept).to(DEV), budget
    c.new.copy_(torch.from_numpy(new))
    ref, before = c.expect(kept), c.score.clone()
    c.compact(A, score)
    assert A.attn_get_device_status() == 0
    assert np.array_equal(c.kc.cpu().numpy(), ref[0]) and np.array_equal(c.vc.cpu().numpy(), ref[1])
    assert np.array_equal(c.score.cpu().numpy(), ref[2] if score else before.cpu().numpy())


@pytest.mark.gpu
def test_bad_lengths_pages_and_entries(A):
    bad = A.ATTN_ERR_DEVICE_BAD_INDEX
    for value in (-5, 10**6):
        c = Cache([50, 60, 70], 2, 32, 8, seed=3)
        c.lend[1] = value
        c.select(A, 20, 2, 4)
        assert A.attn_get_device_status() == bad
        assert (c.kept[1] == -1).all() and c.new.tolist() == [20, value, 20]
        assert (c.kept[0] >= 0).all() and (c.kept[2] >= 0).all()
        before = c.kc.clone()
        c.compact(A)
        own = torch.from_numpy(c.pt[1, :8].astype(np.int64)).to(DEV)
        assert torch.equal(c.kc[own], before[own]) and A.attn_get_device_status() == 0
    for value in (-1, 10**6):  # a page of nobody: its tokens count as less than every score, and are not moved
        c = Cache([50], 2, 32, 8, seed=3, values="all")
        c.ptd[0, 2] = value
        c.select(A, 30, 0, 4)
        assert A.attn_get_device_status() == bad
        got = c.kept.cpu().numpy()
        assert not ((got >= 16) & (got < 24)).any()  # 46 tokens for 26 places: none of those eight
        before = c.kc.clone()
        c.compact(A)  # slots 16 .. 23 lie on that page
        assert A.attn_get_device_status() == bad
        assert torch.equal(c.kc[c.pt[0, 2]], before[c.pt[0, 2]])
    c = Cache([50], 1, 32, 8, seed=4)
    c.select(A, 20, 0, 20)
    c.kept[0, 0, 5], c.kept[0, 0, 6] = 3, c.width * c.page  # below its slot, beyond the table
    want = c.kept.cpu().numpy().copy()
    want[0, 0, 5:7] = -1
    ref = c.expect(want)
    c.compact(A)
    assert A.attn_get_device_status() == bad
    assert np.array_equal(c.kc.cpu().numpy(), ref[0])


@pytest.mark.gpu
def test_streams_and_graph(A):
    """Two captured evictions replayed at once on two streams, on new scores and lengths."""
    cs = [Cache([700, 90, 1500], 4, 64, 16, fmt, seed=5) for fmt in ("bf16", "e4m3")]
    state = [[x.clone() for x in (c.kc, c.vc, c.score)] for c in cs]
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for c in cs:
        c.select(A, 300, 4, 50)
        c.compact(A)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            A.attn_kv_select_paged(c.score, c.ptd, c.lend, c.kept, c.new, 16, c.B, 4, c.width, c.num, 300, 4, 50)
            c.compact(A)
        graphs.append(g)
    for turn in range(3):
        for c, s in zip(cs, state):
            for x, y in zip((c.kc, c.vc, c.score), s):
                x.copy_(y)
            c.score.add_(torch.rand_like(c.score) * turn)
            c.lens[2] -= turn
            c.lend.copy_(torch.from_numpy(c.lens.astype(np.int32)))
        score = [c.score.cpu().numpy() for c in cs]
        want = [np.stack([[wanted(s[c.place(b, np.arange(n))[0], h, c.place(b, np.arange(n))[1]], int(n), 300, 4, 50) for h in range(4)]
                          for b, n in enumerate(c.lens)]) for c, s in zip(cs, score)]
        refs = [c.expect(w) for c, w in zip(cs, want)]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, w, ref in zip(cs, want, refs):
            assert np.array_equal(c.kept.cpu().numpy(), w)
            for got, r in zip((c.kc, c.vc, c.score), ref):
                assert np.array_equal(got.cpu().numpy(), r)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
def test_cache_offsets_beyond_32_bits(A):
    """The last pages of a cache of more than 2^31 elements."""
    Hkv, d, page = 8, 128, 16
    c = Cache([60, 200], Hkv, d, page, seed=6)
    num = 2**31 // (page * Hkv * d) + 9
    far = num - 1 - torch.arange(c.num, device=DEV)
    big = [torch.empty((num, page, Hkv, d), dtype=torch.int16, device=DEV) for _ in range(2)]
    score = torch.zeros((num, Hkv, page), device=DEV)
    big[0][far], big[1][far], score[far] = c.kc, c.vc, c.score
    pt = torch.where((c.ptd >= 0) & (c.ptd < c.num), num - 1 - c.ptd, c.ptd)
    c.select(A, 50, 2, 10)
    kept, new = torch.empty_like(c.kept), torch.empty_like(c.new)
    A.attn_kv_select_paged(score, pt, c.lend, kept, new, page, 2, Hkv, c.width, num, 50, 2, 10)
    assert torch.equal(kept, c.kept) and torch.equal(new, c.new)
    c.compact(A)
    A.attn_kv_compact_paged(*big, score, kept, new, pt, page, 2, Hkv, d, c.width, num, 50, "bf16")
    assert torch.equal(big[0][far], c.kc) and torch.equal(big[1][far], c.vc) and torch.equal(score[far], c.score)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_with_eviction(A, fmt, captured):
    """A serving loop: norms and rotation, cache write, attention, weights, and an eviction whenever a sequence outgrows the budget; against
    the same loop on lists of rows in 64 bits. The choice is taken from the call (its scores carry the attention's rounding) and
    checked against the sums that the call itself holds."""
    B, Hq, Hkv, d, page, budget, sinks, recent, steps, room = 3, 8, 2, 64, 4, 24, 2, 6, 20, 30
    G, scale, eps = Hq // Hkv, 1 / math.sqrt(64), 1e-6
    rs = np.random.RandomState(7)
    width = -(-room // page)
    pt = torch.from_numpy(rs.permutation(B * width).reshape(B, width).astype(np.int32)).to(DEV)
    num = B * width
    kds = vds = 1.0 if fmt == "bf16" else 0.03125  # a power of two: codes times it are exact
    kc, vc = (torch.zeros((num, page, Hkv, d), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device=DEV) for _ in range(2))
    score = torch.full((num, Hkv, page), float("nan"), device=DEV)  # (slots are not cleared, here or later)
    inv = torch.tensor(A.attn_rope_freqs(d)[0], dtype=torch.float64, device=DEV)
    wq, wk = (torch.rand(d, device=DEV) + 0.5 for _ in range(2))
    lens, new = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    qkv = torch.empty((B, (Hq + 2 * Hkv) * d), dtype=torch.bfloat16, device=DEV)
    q, o = (torch.empty((B, Hq, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, lse = torch.empty((B, Hkv, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, Hq), device=DEV)
    kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device=DEV)
    W = qkv.stride(0)

    def step():
        lens.add_(1)
        A.attn_qk_norm_rope(qkv, qkv[:, Hq * d:], q, k, wq, wk, eps, pos, inv, B, Hq, Hkv, d, 0, d, W, W, Hq * d, Hkv * d)
        A.attn_kv_write_paged(k, qkv[:, (Hq + Hkv) * d:], Hkv * d, W, kc, vc, pt, lens, None, page, B, B, Hkv, d, width, num, fmt, kds, vds)
        A.attn_decode_paged_tree(q, kc, vc, pt, lens, None, None, 0, page, o, lse, None, B, B, 1, Hq, Hkv, d, width, num, scale, 0, fmt, kds, vds)
        A.attn_kv_score_paged(q, lse, kc, score, pt, lens, None, page, B, B, 1, Hq, Hkv, d, width, num, scale, 1.0, fmt, kds)
        pos.add_(1)

    def evict():
        A.attn_kv_select_paged(score, pt, lens, kept, new, page, B, Hkv, width, num, budget, sinks, recent)
        A.attn_kv_compact_paged(kc, vc, score, kept, new, pt, page, B, Hkv, d, width, num, budget, fmt)
        lens.copy_(new)

    def rows(x, b, h, n):
        t = np.arange(n)
        y = x[pt[b, t // page].long(), torch.from_numpy(t % page).to(DEV), h]
        return y.double() if fmt == "bf16" else y.view(torch.float8_e4m3fn).double() * kds

    keys = [[[] for _ in range(Hkv)] for _ in range(B)]  # rows as cached, and their sums, in the order of the slots
    vals = [[[] for _ in range(Hkv)] for _ in range(B)]
    sums = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]
    run, drop = step, evict
    if captured:
        qkv.normal_()
        step()
        evict()
        graphs = []
        for f in (step, evict):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            graphs.append(g)
        run, drop = graphs[0].replay, graphs[1].replay
        lens.zero_(), pos.zero_()
    start = [1, 15, 23]
    for i in range(steps + max(start)):
        active = [i >= max(start) - s for s in start]  # sequences that have not begun write their slot 0 over and over
        for b in range(B):
            if not active[b]:
                lens[b] = 0
                pos[b] = 0
                keys[b], vals[b] = [[] for _ in range(Hkv)], [[] for _ in range(Hkv)]
                sums[b] = [np.zeros(0) for _ in range(Hkv)]
        qkv.copy_(torch.from_numpy(rs.standard_normal(tuple(qkv.shape))))
        run()
        ns = lens.tolist()
        for b in range(B):
            for h in range(Hkv):
                n = ns[b]
                K, V = rows(kc, b, h, n), rows(vc, b, h, n)
                keys[b][h].append(K[n - 1])
                vals[b][h].append(V[n - 1])
                assert torch.equal(K, torch.stack(keys[b][h])) and torch.equal(V, torch.stack(vals[b][h]))  # nothing lost or mixed up
                s = (q[b, h * G:(h + 1) * G].double() @ K.T) * scale
                p = s.softmax(-1)
                # O and LSE within the library's bar for the attention; a weight within the LSE's 2e-3
                assert ((p @ V) - o[b, h * G:(h + 1) * G].double()).abs().max() <= 1.5e-2 + 2.0**-7 * V.abs().max()
                sums[b][h] = np.append(sums[b][h], 0.0) + p.sum(0).cpu().numpy()
                t = np.arange(n)
                got = score[pt[b, t // page].long(), h, torch.from_numpy(t % page).to(DEV)].double().cpu().numpy()
                assert (np.abs(got - sums[b][h]) <= 2.1e-3 * sums[b][h] + 1e-9).all()
        if i % 3 == 2:
            held = score.cpu().numpy()
            drop()
            for b in range(B):
                for h in range(Hkv):
                    t = np.arange(ns[b])
                    row = kept[b, h].cpu().numpy()
                    assert np.array_equal(row, wanted(held[pt[b].cpu().numpy()[t // page], h, t % page], ns[b], budget, sinks, recent))
                    row = row[row >= 0]
                    keys[b][h], vals[b][h] = [keys[b][h][x] for x in row], [vals[b][h][x] for x in row]
                    sums[b][h] = sums[b][h][row]
            assert lens.tolist() == [min(n, budget) for n in ns]
    assert A.attn_get_device_status() == 0 and max(ns) >= budget


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 300])
def test_calls_behind_one_another(A, fmt, n):
    """Each call reads what the one before it writes, and may start before that has ended: the same bytes with the device idle in between."""
    B, Hq, Hkv, d, page, budget, length = 24, 8, 2, 128, 16, 160, 600
    W, T, width = (Hq + 2 * Hkv) * d, B * n, -(-length // page)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn((T, W), generator=g, device=DEV).bfloat16()
    pt = torch.randperm(B * width, generator=g, device=DEV).int().view(B, width)
    shape = (B * width, page, Hkv, d)
    cache = [torch.randn(shape, generator=g, device=DEV).bfloat16() if fmt == "bf16" else
             torch.randn(shape, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    sums = torch.rand((B * width, Hkv, page), generator=g, device=DEV)
    lens = torch.full((B,), length, dtype=torch.int32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv = torch.tensor(A.attn_rope_freqs(d)[0], dtype=torch.float64, device=DEV)
    w = torch.rand(d, generator=g, device=DEV) + 0.5
    lse = torch.rand((T, Hq), generator=g, device=DEV) + 5
    dy = torch.randn((T, Hq * d), generator=g, device=DEV).bfloat16()

    def run(between):
        kc, vc, score = cache[0].clone(), cache[1].clone(), sums.clone()
        q, dq = torch.zeros((2, T, Hq, d), dtype=torch.bfloat16, device=DEV)
        k, dw = torch.zeros((T, Hkv, d), dtype=torch.bfloat16, device=DEV), torch.zeros(d, device=DEV)
        kept, new = torch.zeros((B, Hkv, budget), dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
        for call in (
                lambda: A.attn_qk_norm_rope(x, x[:, Hq * d:], q, k, w, w, 1e-6, pos, inv, T, Hq, Hkv, d, 0, d, W, W, Hq * d, Hkv * d),
                lambda: A.attn_qk_norm_rope_bwd(q, None, dy, None, w, None, 1e-6, pos, inv, dq, None, dw, None, T, Hq, 0, d, 0, d, Hq * d, 0,
                                                Hq * d, 0, Hq * d, 0),
                lambda: A.attn_kv_write_paged(k, x[:, (Hq + Hkv) * d:], Hkv * d, W, kc, vc, pt, lens, None, page, T, B, Hkv, d, width, B * width, fmt),
                lambda: A.attn_kv_score_paged(q, lse, kc, score, pt, lens, None, page, T, B, n, Hq, Hkv, d, width, B * width, 0.1, 0.5, fmt),
                lambda: A.attn_kv_score_paged(dq, lse, kc, score, pt, lens, None, page, T, B, n, Hq, Hkv, d, width, B * width, 0.1, 0.5, fmt),
                lambda: A.attn_kv_select_paged(score, pt, lens, kept, new, page, B, Hkv, width, B * width, budget, 4, 16),
                lambda: A.attn_kv_compact_paged(kc, vc, score, kept, new, pt, page, B, Hkv, d, width, B * width, budget, fmt),
                lambda: A.attn_kv_score_paged(q[:B], lse[:B], kc, score, pt, new, None, page, B, B, 1, Hq, Hkv, d, width, B * width, 0.1, 1.0, fmt)):
            call()
            between()
        return q, k, dq, dw, kc, vc, score, kept, new

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a, b)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hkv,budget,sinks,recent", [([1000], 2, 256, 4, 32), ([10, 0, 3000, 64, 65], 3, 64, 4, 8), ([9000, 40], 1, 8000, 0, 100)])
@pytest.mark.parametrize("page,tokens", [(16, 131072), (7, 131068), (16, 2**20)])
@pytest.mark.parametrize("values", ["sums", "few", "all"])
def test_short_sequences_in_a_wide_table(A, lens, Hkv, budget, sinks, recent, page, tokens, values):
    """A page table for far longer contexts (several blocks share a row, or the keys are read again for every step), most parts of it empty."""
    c = Cache(lens, Hkv, 16, page, values=values)
    c.ptd = torch.nn.functional.pad(c.ptd, (0, tokens // page - c.width), value=-1).contiguous()
    c.width = tokens // page
    c.select(A, budget, sinks, recent)
    assert A.attn_get_device_status() == 0
    score = c.score.cpu().numpy()
    want = np.stack([[wanted(score[c.place(b, np.arange(n))[0], h, c.place(b, np.arange(n))[1]], int(n), budget, sinks, recent)
                      for h in range(Hkv)] for b, n in enumerate(c.lens)])
    assert np.array_equal(c.kept.cpu().numpy(), want)
    expect = c.expect(want)
    c.compact(A)
    assert A.attn_get_device_status() == 0
    for got, ref in zip((c.kc, c.vc, c.score), expect):
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=got.dtype == torch.float32)


@pytest.mark.gpu
def test_the_largest_budget(A):
    """A budget of 2^31 - 1: one short row and all entries behind it; then a length out of range, whose slots up to 2^31 - 1 are all looked at
    and left alone."""
    budget = 2**31 - 1
    c = Cache([50, 20], 1, 16, 8, seed=17)
    c.B, c.lend = 1, c.lend[:1].clone()
    c.select(A, budget, 3, 2**31 - 100)
    assert A.attn_get_device_status() == 0 and c.new[0] == 50
    assert torch.equal(c.kept[0, 0, :50], torch.arange(50, dtype=torch.int32, device=DEV))
    assert all((c.kept[0, 0, i:min(i + 2**28, budget)] == -1).all() for i in [50] + list(range(2**28, budget, 2**28)))
    before = c.kc.clone()
    c.compact(A)
    assert torch.equal(c.kc, before) and A.attn_get_device_status() == 0
    c.lend[0] = budget
    c.kept.fill_(-9)
    A.attn_kv_select_paged(c.score, c.ptd, c.lend, c.kept, c.new, c.page, 1, 1, c.width, c.num, budget, 3, 4)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_BAD_INDEX and c.new[0] == budget
    assert all((c.kept[0, 0, i:min(i + 2**28, budget)] == -1).all() for i in range(0, budget, 2**28))
    c.compact(A)
    assert torch.equal(c.kc, before) and A.attn_get_device_status() == 0
