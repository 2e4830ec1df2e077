"""attn_decode_paged_tree: refusals on the CPU; on the GPU every row and head against 64-bit
arithmetic with a bound that counts the roundings, over formats, head layouts, lengths, page sizes,
masks that leave rows empty, and slots that hold anything."""
import math

import numpy as np
import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")
DEV = "cuda:0"
BIG = {"e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(scope="module")
def A():
    ensure_built()
    import exact_softmax_attention_gb300 as mod
    return mod


# ------------------------------------------------------------------------------------- CPU

def status(A, **kw):
    a = dict(q=0x1000, k_cache=0x2000, v_cache=0x3000, page_table=0x4000, seqlens=0x5000, cu_seqlens=None, tree_mask=0x6000,
             mask_words=1, page_size=16, o=0x7000, lse=0x8000, stream=0, T=0, B=1, max_q=8, Hq=8, Hkv=2, d=128,
             max_pages_per_seq=4, num_pages=8, scale=0.1, num_splits=0, kv_format="e4m3", k_descale=0.5, v_descale=2.0)
    a.update(kw)
    return A.attn_decode_paged_tree(**a, raise_on_error=False)


def test_refusals(A):
    null, shape, align, arg = A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    assert status(A) == A.ATTN_OK and status(A, B=0) == A.ATTN_OK and status(A, tree_mask=None, mask_words=9) == A.ATTN_OK
    for name in ("q", "k_cache", "v_cache", "page_table", "seqlens", "o", "lse"):
        assert status(A, **{name: None}) == null
    for bad in (dict(T=-1), dict(B=-1), dict(B=65536), dict(max_q=0), dict(max_q=257, mask_words=4), dict(max_q=65), dict(mask_words=0),
                dict(mask_words=5), dict(Hq=0), dict(Hq=9), dict(Hkv=0), dict(d=96), dict(page_size=0), dict(max_pages_per_seq=0),
                dict(num_pages=0), dict(num_splits=-1), dict(T=9, B=2), dict(T=9, B=1), dict(T=4, B=0),
                dict(num_pages=1 << 27), dict(max_pages_per_seq=1 << 27), dict(scale=float("nan")),
                dict(max_q=64, Hq=2048, Hkv=1)):
        assert status(A, **bad) == shape, bad
    for bad in (dict(kv_format=3), dict(k_descale=float("nan")), dict(v_descale=float("inf")), dict(scale=1e30, k_descale=1e30)):
        assert status(A, **bad) == arg, bad
    for bad in (dict(q=0x1008), dict(o=0x7008), dict(k_cache=0x2001), dict(v_cache=0x3008), dict(lse=0x8002), dict(page_table=0x4001),
                dict(seqlens=0x5002), dict(cu_seqlens=0x9002), dict(tree_mask=0x6004)):
        assert status(A, **bad) == align, bad


# ------------------------------------------------------------------------------------- GPU

def random_tree(rs, n):
    """Ancestor bits of a random tree of n nodes, each node's parent one before it (or the context)."""
    seen = np.zeros((n, n), bool)
    for i in range(n):
        p = rs.randint(-1, i) if i else -1
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return seen


class Case:
    """n[b] drafted of lens[b] cached tokens; tree: "tree", "chain", "any" (random bits, some rows
    empty), "none" (no drafted token sees any)."""

    def __init__(self, fmt, Hq, Hkv, d, page, n, lens, tree="tree", seed=0, dense=False, qmult=1.0, tail=2):
        rs = np.random.RandomState(seed)
        self.fmt, self.Hq, self.Hkv, self.d, self.page, self.n, self.lens, self.dense = fmt, Hq, Hkv, d, page, n, lens, dense
        self.B, self.T = len(n), sum(n) + (0 if dense else tail)
        self.max_q = max(1, max(n))
        pages = [-(-l // page) for l in lens]
        self.num, self.width = sum(pages) + 2, max(1, max(pages))
        perm, at = rs.permutation(self.num), 0
        self.pt = np.full((self.B, self.width), 2**31 - 1, np.int32)  # unused entries are never read
        for b, c in enumerate(pages):
            self.pt[b, :c] = perm[at:at + c]
            at += c
        shape = (self.num, page, Hkv, d)
        self.ds = (1.0, 1.0) if fmt == "bf16" else (0.02, 0.03)
        x = torch.from_numpy(rs.standard_normal((2, *shape)).astype(np.float32))
        if fmt == "bf16":
            self.c = [y.bfloat16().to(DEV) for y in x]
        else:
            t = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
            self.c = [(y / s).to(t).view(torch.uint8).to(DEV) for y, s in zip(x, self.ds)]
        self.q = (torch.from_numpy(rs.standard_normal((self.T, Hq, d))) * qmult).bfloat16().to(DEV)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.seen = [np.tril(np.ones((m, m), bool)) if tree == "chain" else np.zeros((m, m), bool) if tree == "none"
                     else rs.rand(m, m) < 0.2 if tree == "any" else random_tree(rs, m) for m in n]
        self.words = -(-self.max_q // 64)
        bits = np.full((self.T, self.words), 2**64 - 1, np.uint64)  # bits at and above n are ignored
        for b, m in enumerate(n):
            for i in range(m):
                v = (2**(64 * self.words) - 1) >> m << m
                for j in range(m):
                    v |= int(self.seen[b][i, j]) << j
                for w in range(self.words):
                    bits[self.cu[b] + i, w] = (v >> (64 * w)) & (2**64 - 1)
        self.mask = None if tree == "chain" else torch.from_numpy(bits.view(np.int64)).to(DEV)
        self.scale = 1.0 / math.sqrt(d)
        self.dev = {"pt": torch.from_numpy(self.pt).to(DEV), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
                    "cu": None if dense else torch.from_numpy(self.cu).to(DEV)}
        self.o = torch.full((self.T, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, Hq), 7.0, dtype=torch.float32, device=DEV)

    def run(self, A, num_splits=0, scale=None, stream=None):
        d = self.dev
        A.attn_decode_paged_tree(self.q, self.c[0], self.c[1], d["pt"], d["lens"], d["cu"], self.mask, self.words, self.page, self.o,
                                 self.lse, stream, self.T, self.B, self.max_q, self.Hq, self.Hkv, self.d, self.width, self.num,
                                 self.scale if scale is None else scale, num_splits, self.fmt, *self.ds)

    def values(self):
        out = []
        for c, s in zip(self.c, self.ds):
            v = c if self.fmt == "bf16" else c.view(torch.float8_e4m3fn if self.fmt == "e4m3" else torch.float8_e5m2)
            out.append(v.double().cpu().numpy().reshape(-1, self.Hkv, self.d) * float(np.float32(s)))
        return out

    def reference(self, scale=None):
        """(o, lse, bound of o, bound of lse) in 64 bits; rows that see nothing: 0, -inf."""
        scale = self.scale if scale is None else float(np.float32(scale))
        K, V = self.values()
        q = self.q.double().cpu().numpy()
        o, lse = np.zeros((self.T, self.Hq, self.d)), np.full((self.T, self.Hq), -np.inf)
        bo, bl = np.zeros_like(o), np.zeros_like(lse)
        G = self.Hq // self.Hkv
        for b, (m, l) in enumerate(zip(self.n, self.lens)):
            at = np.arange(l)
            rows = self.pt[b, at // self.page].astype(np.int64) * self.page + at % self.page
            vis = np.ones((m, l), bool)
            if l:
                vis[:, l - m:] = self.seen[b]
            for i in range(m):
                keys = rows[vis[i]] if l else rows
                if not len(keys):
                    continue
                for h in range(self.Hq):
                    k, v, x = K[keys, h // G], V[keys, h // G], q[self.cu[b] + i, h]
                    s = k @ x * scale
                    z = s.max() + np.log(np.exp(s - s.max()).sum())
                    w = np.exp(s - z)
                    o[self.cu[b] + i, h], lse[self.cu[b] + i, h] = w @ v, z
                    aw = w @ np.abs(v)
                    # fp32 scores (d products and sums), the exponent's argument and 2^x (2^-21 together
                    # with |s| 2^-23 for s log2 e), and the sums over the keys
                    e = (np.abs(k) @ np.abs(x)).max() * abs(scale) * (self.d + 4) * 2.0**-24 + 2.0**-20 + np.abs(s).max() * 2.0**-22 \
                        + (len(keys) / 16 + 40) * 2.0**-24
                    if self.fmt != "bf16":  # q as two e4m3 parts: elements off by at most 2^-17 of the row's largest
                        e += np.abs(x).max() * 2.0**-17 * np.abs(k).sum(1).max() * abs(scale)
                    p_step = 2.0**-8 if self.fmt == "bf16" else 2.0**-11  # half a step of P, relative
                    small = 0.0 if self.fmt == "bf16" else len(keys) * 2.0**-25 * np.abs(v).max()  # f16 below its normal range
                    bo[self.cu[b] + i, h] = aw * (p_step + 2 * e) + small
                    bl[self.cu[b] + i, h] = e + abs(z) * 2.0**-22
        bo += 2.0**-8 * (np.abs(o) + bo)  # the rounding of the output
        return o, lse, bo + 1e-30, bl

    def check(self, scale=None):
        ro, rl, bo, bl = self.reference(scale)
        n = sum(self.n)
        o, lse = self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(lse[:n]), np.isneginf(rl[:n]))
        assert np.isfinite(o[:n]).all()
        do = np.abs(o[:n] - ro[:n]) / bo[:n]
        assert (do <= 1).all(), f"o: {do.max():.3f} of the bound"
        f = np.isfinite(rl[:n])
        dl = np.abs(lse[:n][f] - rl[:n][f]) / bl[:n][f]
        assert (dl <= 1).all(), f"lse: {dl.max():.3f} of the bound"
        assert (o[n:] == 7).all() and (lse[n:] == 7).all()  # rows behind the last sequence


CASES = {
    "one_row": ("bf16", 1, 1, 128, 16, [1], [1], "chain"),
    "gqa4_n4": ("bf16", 8, 2, 128, 16, [4, 4, 4], [4, 300, 1000], "tree"),
    "d64_p7": ("bf16", 6, 2, 64, 7, [5, 1, 3], [5, 64, 500], "tree"),
    "n8_g4": ("bf16", 8, 2, 128, 16, [8, 0, 7, 8], [1024, 5, 63, 65], "tree"),
    "n16_g8": ("bf16", 16, 2, 128, 64, [16, 16], [700, 2000], "tree"),
    "n33_g4": ("bf16", 4, 1, 128, 16, [33, 20, 1], [33, 800, 129], "tree"),
    "n64_g4": ("bf16", 8, 2, 128, 16, [64, 63], [64, 900], "any"),
    "n70_g3": ("bf16", 3, 1, 128, 1, [70, 65, 2], [70, 401, 500], "tree"),
    "n256_g1": ("bf16", 1, 1, 64, 32, [256, 129], [256, 400], "any"),
    "n200_chain": ("bf16", 2, 1, 128, 16, [200, 1], [500, 1], "chain"),
    "none": ("bf16", 4, 2, 128, 16, [5, 20], [5, 100], "none"),
    "mqa_g40": ("bf16", 40, 1, 64, 16, [3, 2], [300, 2], "tree"),
    "e4m3_n3": ("e4m3", 8, 2, 128, 16, [3, 3], [600, 3], "tree"),
    "e4m3_n16": ("e4m3", 8, 2, 128, 16, [16, 16, 9], [16, 1000, 130], "tree"),
    "e4m3_n48_d64": ("e4m3", 4, 1, 64, 5, [48, 17], [48, 333], "any"),
    "e5m2_n5_d64": ("e5m2", 12, 3, 64, 7, [5, 1, 4, 0], [900, 1, 4, 9], "chain"),
    "e5m2_n64": ("e5m2", 8, 1, 128, 16, [64], [700], "tree"),
    "e4m3_n130": ("e4m3", 2, 2, 128, 1000, [130], [1500], "tree"),
    "zero_lengths": ("e4m3", 4, 2, 128, 16, [4, 2, 0], [0, 2, 0], "tree"),
    "zero_lengths_many_rows": ("bf16", 8, 1, 64, 16, [30, 30], [0, 30], "tree"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("num_splits", [0, 1, 5])
def test_parity(A, name, num_splits):
    c = Case(*CASES[name], seed=len(name))
    c.run(A, num_splits)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 24])
def test_dense_rows_need_no_offsets(A, fmt, n):
    c = Case(fmt, 4, 2, 128, 16, [n] * 3, [n, 90, 400], "tree", 5, dense=True)
    c.run(A)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0, 1e-46])
def test_any_finite_scale(A, n, scale):
    """Negative and zero scales (a plain product with -inf would be +inf or NaN), and sharp ones."""
    c = Case("bf16", 4, 2, 64, 16, [n, n], [n + 3, 300], "any", 6)
    c.run(A, 2, scale)
    assert A.attn_get_device_status() == 0
    c.check(scale)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d", [("bf16", 3, 128), ("e5m2", 3, 64), ("bf16", 37, 64), ("e5m2", 37, 128), ("e4m3", 37, 128)])
@pytest.mark.parametrize("num_splits", [1, 4])
def test_masked_slots_hold_anything(A, fmt, n, d, num_splits):
    """NaN (and infinities) in unused slots of the last page and in drafted tokens nobody sees."""
    c = Case(fmt, 4, 2, d, 16, [n, n], [n + 61, 300 + n], "tree", 7)
    dead = n // 2
    for s in c.seen:
        s[:, dead] = False
    m = c.mask.cpu().numpy().view(np.uint64)
    m &= ~(np.uint64(1) << np.uint64(dead))
    c.mask = torch.from_numpy(m.view(np.int64)).to(DEV)
    fills = [float("nan"), float("inf")] if fmt == "bf16" else [0x7F, 0x7C] if fmt == "e5m2" else [0x7F]
    for cache in c.c:
        flat = cache.view(-1, c.Hkv, d)
        for b in range(2):
            last = c.lens[b] - 1
            page = int(c.pt[b, last // 16]) * 16
            flat[page + last % 16 + 1:page + 16] = fills[0]
            at = c.lens[b] - n + dead
            flat[int(c.pt[b, at // 16]) * 16 + at % 16] = fills[-1]
        used = c.pt[c.pt < c.num]
        for page in set(range(c.num)) - set(used.tolist()):
            cache[page] = fills[0]
    c.run(A, num_splits)
    assert A.attn_get_device_status() == 0
    keep = c.values
    c.values = lambda: [np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in keep()]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 37])
@pytest.mark.parametrize("where", ["drafted", "context"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_visible_nonfinite_values_stay(A, n, where, value):
    """A non-finite V element reaches exactly the rows that see its token, and only its column."""
    c = Case("bf16", 4, 2, 64, 16, [n], [n + 70], "tree", 8)
    tok = (69 if where == "context" else 70 + 1)
    row = int(c.pt[0, tok // 16]) * 16 + tok % 16
    c.c[1].view(-1, 2, 64)[row, 1, 5] = value
    c.run(A, 3)
    o = c.o.double().cpu().numpy()
    hit = np.zeros((c.T, 4, 64), bool)
    rows = np.ones(n, bool) if where == "context" else c.seen[0][:, 1]
    hit[:n][rows, 2:, 5] = True
    assert np.array_equal(~np.isfinite(o), hit)
    assert (np.isposinf(o[hit]) if value == float("inf") else np.isnan(o[hit])).all()


def shortest(f, calls=10, rounds=6):
    """Least time of a call among others, in us."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    best = math.inf
    for _ in range(rounds):
        ev[0].record()
        for _ in range(calls):
            f()
        ev[1].record()
        ev[1].synchronize()
        best = min(best, ev[0].elapsed_time(ev[1]) * 1e3 / calls)
    return best


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d,page", [("bf16", 16, 128, 16), ("e4m3", 16, 128, 64), ("e5m2", 40, 64, 64), ("bf16", 4, 128, 64)])
def test_unused_slots_cost_nothing(A, fmt, n, d, page):
    """NaN behind the last token of every sequence: the work is the same as over zeros there, and so is the time (half as
    much again and 5 us are for the clock; a search for rows that see them took a millisecond or more)."""
    times = []
    for fill in (0, float("nan") if fmt == "bf16" else 0x7F):
        c = Case(fmt, 8, 2, d, page, [n] * 4, [n + 900 + 3 * i for i in range(4)], "tree", 7)
        for cache in c.c:
            for b, l in enumerate(c.lens):
                at = int(c.pt[b, (l - 1) // page]) * page
                cache.view(-1, 2, d)[at + (l - 1) % page + 1:at + page] = fill
        times.append(shortest(lambda: c.run(A)))
        c.check()
    assert times[1] <= 1.5 * times[0] + 5, times


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d,page", [("bf16", 16, 128, 16), ("e4m3", 64, 128, 64), ("e5m2", 200, 64, 64), ("bf16", 256, 64, 7),
                                          ("bf16", 4, 128, 64), ("e4m3", 8, 64, 7)])
@pytest.mark.parametrize("where", ["a masked token", "every drafted token"])
def test_time_of_nonfinite_drafted_values(A, fmt, n, d, page, where):
    """Non-finite values of drafted tokens, that no row sees or that most do: at most one pass over the 64-token tiles
    that hold drafted tokens, read once per warp of rows. 64 rows of V in loads eight at a time (2 us each with the look-ups), and,
    where they are seen, 32 rows of outputs read and written at 1 us: 50 us a tile at most. (Row by row, column by column
    and token by token it took milliseconds.)"""
    times = []
    for fill in (0, float("nan") if fmt == "bf16" else 0x7F):
        c = Case(fmt, 8, 2, d, page, [n] * 4, [n + 900 + 3 * i for i in range(4)], "tree", 7)
        for b, l in enumerate(c.lens):
            for t in [l - n // 2] if where == "a masked token" else range(l - n, l):
                c.c[1].view(-1, 2, d)[int(c.pt[b, t // page]) * page + t % page] = fill
        if where == "a masked token":
            m = c.mask.cpu().numpy().view(np.uint64)
            m[:, (n - n // 2) // 64] &= ~(np.uint64(1) << np.uint64((n - n // 2) % 64))
            c.mask = torch.from_numpy(m.view(np.int64)).to(DEV)
        times.append(shortest(lambda: c.run(A), 3))
    tiles = 1 if where == "a masked token" else (n + 63) // 64 + 1
    assert times[1] <= 1.5 * times[0] + 50 * tiles, times


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("bf16", 3), ("e5m2", 3), ("bf16", 37), ("e5m2", 37)])
@pytest.mark.parametrize("num_splits", [1, 2, 8, 20])
def test_infinities_of_both_signs(A, fmt, n, num_splits):
    """-inf in a context token of a tile that every row sees in full, +inf in a drafted one (in the same split or
    another): inf - inf is NaN in the rows that see both, -inf in the others."""
    c = Case(fmt, 4, 2, 64, 16, [n], [n + 700], "tree", 8)
    for tok, value, code in ((600, -math.inf, 0xFC), (700 + 1, math.inf, 0x7C)):
        row = int(c.pt[0, tok // 16]) * 16 + tok % 16
        c.c[1].view(-1, 2, 64)[row, 1, 5] = value if fmt == "bf16" else code
    c.run(A, num_splits)
    assert A.attn_get_device_status() == 0
    o = c.o[:n].float().cpu().numpy()
    both = c.seen[0][:, 1]
    assert both.any() and not both.all()
    assert np.isnan(o[both, 2:, 5]).all() and np.isneginf(o[~both, 2:, 5]).all()
    o[:, 2:, 5] = 0
    assert np.isfinite(o).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("e4m3", 3), ("e4m3", 30), ("e5m2", 30), ("bf16", 30)])
def test_queries_of_any_range(A, fmt, n):
    """Rows of q scaled from 2^-100 to 2^12, with elements spread over 2^20 within a row, zero rows, and scores
    that a small scale brings back into range."""
    c = Case(fmt, 4, 2, 128, 16, [n, n], [n, 250], "tree", 21)
    rs = np.random.RandomState(3)
    spread = torch.from_numpy(2.0 ** rs.randint(-20, 1, c.q.shape)).to(DEV)
    c.q.copy_((c.q.double() * spread).bfloat16())
    c.q[0] *= 2.0**-100 if fmt == "bf16" or n > 16 else 2.0**-10  # up to 16 rows q passes through f16
    c.q[1] *= 2.0**12
    c.q[2, 1] = 0
    c.run(A, 2, 2.0**-12)
    assert A.attn_get_device_status() == 0
    c.check(2.0**-12)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("n,d,wide", [(1, 128, 1), (3, 128, 1), (3, 64, 1), (6, 64, 1), (6, 64, 4000), (2, 64, 1)])
@pytest.mark.parametrize("power", [-100, -40, 20, 100])
def test_queries_of_any_range_in_few_rows(A, fmt, n, d, wide, power):
    """8-bit caches: what q may be does not depend on the number of rows or on the width of the table. Rows of 2^power,
    one 2^8 above and one of zeros, elements spread over 2^20 within a row, and the scale that brings them back."""
    c = widened(Case(fmt, 8, 2, d, 16, [n, n], [n + 250, n + 40], "tree", 21), wide)
    rs = np.random.RandomState(4)
    c.q.copy_((c.q.double() * torch.from_numpy(2.0 ** (power - rs.randint(0, 20, c.q.shape).astype(float))).to(DEV)).bfloat16())
    c.q[0, 2] *= 2.0**8
    c.q[0, 3] = 0
    scale = 2.0 ** (-power - 2)
    c.run(A, 0, scale)
    assert A.attn_get_device_status() == 0
    c.check(scale)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d", [("e4m3", 3, 128), ("e5m2", 6, 64), ("e4m3", 30, 64), ("bf16", 3, 128), ("bf16", 30, 128)])
def test_large_queries_on_zero_keys(A, fmt, n, d):
    """Scores of 0 from factors whose product leaves fp32: a plain mean over what each row sees."""
    c = Case(fmt, 4, 1, d, 16, [n], [n + 70], "any", 25)
    c.q.fill_(2.0**125)
    c.c[0].zero_()
    c.run(A, 2, 2.0**120 if fmt == "bf16" else 2.0**125)
    assert A.attn_get_device_status() == 0
    c.check(1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("e4m3", 30), ("bf16", 30), ("bf16", 3)])
def test_vanishing_queries_and_scales(A, fmt, n):
    """Scores far below the range of fp32: a plain mean over what each row sees."""
    c = Case(fmt, 4, 2, 64, 16, [n], [n + 70], "any", 25)
    c.q.mul_(2.0**-115)
    c.run(A, 2, 2.0**-60)
    assert A.attn_get_device_status() == 0
    c.check(2.0**-60)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 30])
@pytest.mark.parametrize("threshold", [0.0, 60.0])
def test_any_rescale_threshold(A, fmt, n, threshold):
    """Rescaling on every rise of the maximum, and (nearly) never: both are exact."""
    c = Case(fmt, 4, 2, 128, 16, [n], [600], "tree", 22, qmult=3.0)
    A.attn_set_option("rescale_threshold", threshold)
    try:
        c.run(A, 2)
    finally:
        A.attn_set_option("rescale_threshold", 8.0)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,page", [("bf16", 2, 16), ("bf16", 20, 16), ("bf16", 20, 7), ("e4m3", 3, 16), ("e4m3", 20, 16)])
def test_cache_offsets_beyond_32_bits(A, fmt, n, page):
    """Rows written, read back and attended more than 2^32 bytes (and elements) into the caches."""
    Hkv, d = 8, 128
    c = Case(fmt, 8, Hkv, d, page, [n, n], [n, 120], "tree", 23)
    rows = (1 << 32) // (Hkv * d) + 40 * page
    c.num = rows // page
    t = torch.bfloat16 if fmt == "bf16" else torch.uint8
    small = c.c
    big = [torch.empty((c.num, page, Hkv, d), dtype=t, device=DEV) for _ in range(2)]
    moved = c.pt < 1 << 20
    shift = c.num - small[0].shape[0]  # the case's pages move to the end of the large caches
    for b, s in zip(big, small):
        b[shift:] = s
    c.pt = np.where(moved, c.pt + shift, c.pt).astype(np.int32)
    c.dev["pt"] = torch.from_numpy(c.pt).to(DEV)
    c.c = big
    vals = c.values
    x = torch.randn((c.T, 2 * Hkv * d), device=DEV, dtype=torch.bfloat16)
    k, v = x[:, :Hkv * d], x[:, Hkv * d:]
    A.attn_kv_write_paged(k, v, x.stride(0), x.stride(0), *c.c, c.dev["pt"], c.dev["lens"], c.dev["cu"], page, c.T, c.B, Hkv, d, c.width,
                          c.num, fmt, *c.ds)
    c.run(A, 2)
    back = torch.zeros((2, c.T, Hkv * d), device=DEV, dtype=torch.bfloat16)
    A.attn_kv_read_paged(*c.c, back[0], back[1], Hkv * d, Hkv * d, c.dev["pt"], c.dev["lens"], c.dev["cu"], page, c.T, c.B, Hkv, d,
                         c.width, c.num, fmt, *c.ds)
    assert A.attn_get_device_status() == 0
    m = sum(c.n)
    step = {"bf16": 0.0, "e4m3": 2.0**-4 + 2.0**-8}[fmt]
    assert ((back[1][:m].double() - v[:m].double()).abs() <= v[:m].double().abs() * step * 1.01 + 1e-3 * (step > 0)).all()
    c.c = [b[shift:].clone() for b in big]  # what the reference reads
    c.pt = np.where(moved, c.pt - shift, c.pt).astype(np.int32)
    del big, vals
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 20])
def test_a_slice_of_the_offsets(A, n):
    """Offsets are absolute rows: a call on the later sequences leaves the rows before them alone."""
    c = Case("bf16", 4, 2, 64, 16, [n, n, n], [40, 300, n], "tree", 24)
    c.run(A)
    want = c.o.clone(), c.lse.clone()
    c.o.fill_(7)
    c.lse.fill_(7)
    d = c.dev
    A.attn_decode_paged_tree(c.q, *c.c, d["pt"][1:], d["lens"][1:], d["cu"][1:], c.mask, c.words, 16, c.o, c.lse, None, c.T, 2, c.max_q, 4,
                             2, 64, c.width, c.num, c.scale)
    assert A.attn_get_device_status() == 0
    assert (c.o[:n] == 7).all() and (c.lse[:n] == 7).all()
    assert torch.equal(c.o[n:], torch.cat((want[0][n:3 * n], c.o[3 * n:]))) and (c.o[3 * n:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 30])
def test_nan_query_stays_in_its_rows(A, n):
    c = Case("bf16", 4, 2, 64, 16, [n, n], [n, 200], "tree", 9)
    c.q[1, 2] = float("nan")
    c.run(A, 2)
    bad = torch.isnan(c.lse)
    assert bad[1, 2] and bad.sum() == 1
    assert torch.isnan(c.o[1, 2].float()).all() and torch.isnan(c.o.float()).sum() == 64


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("bf16", 3), ("e4m3", 3), ("bf16", 20), ("e4m3", 20)])
def test_bad_lengths_pages_and_offsets(A, fmt, n):
    bad = A.ATTN_ERR_DEVICE_BAD_INDEX

    def fresh():
        return Case(fmt, 4, 2, 128, 16, [n, n, n], [n, 100, 400], "tree", 11)

    for b, length in ((0, n - 1), (1, -4), (2, 401 + 16 * 100)):
        c = fresh()
        c.dev["lens"][b] = length
        c.run(A)
        assert A.attn_get_device_status() == bad
        c.lens[b] = 0
        c.check()
    c = fresh()  # pages out of range count as zero rows
    c.dev["pt"][2, 3], c.dev["pt"][2, 7] = -1, c.num
    c.run(A, 2)
    assert A.attn_get_device_status() == bad
    ghost = c.num  # two more pages of zeros stand for them
    c.pt[2, 3] = c.pt[2, 7] = ghost
    vals = c.values()
    c.values = lambda: [np.concatenate([x, np.zeros((16, *x.shape[1:]))]) for x in vals]
    c.check()
    c = fresh()  # the last sequence passes the rows, or holds more than max_q of them: its rows stay
    for change in ("rows", "max_q"):
        c = fresh()
        if change == "rows":
            c.dev["cu"][3] = c.T + 1
        else:
            c.dev["cu"][3] += 1
        c.run(A)
        assert A.attn_get_device_status() == bad
        c.n = [n, n]
        c.T, keep = 2 * n, (c.o, c.lse)
        assert (c.o[2 * n:] == 7).all() and (c.lse[2 * n:] == 7).all()
        c.lens, c.B = c.lens[:2], 2
        c.check()


@pytest.mark.gpu
def test_agrees_with_the_one_token_decode(A):
    """One drafted token that sees itself is the decode of one token."""
    c = Case("bf16", 16, 4, 128, 16, [1] * 5, [1, 16, 17, 300, 1500], "chain", 12, dense=True)
    c.run(A)
    o, lse = torch.empty_like(c.o), torch.empty_like(c.lse)
    A.attn_decode_paged(c.q, c.c[0], c.c[1], c.dev["pt"], c.dev["lens"], 16, o, lse, None, c.B, 16, 4, 128, c.width, c.num, c.scale)
    assert (o.float() - c.o.float()).abs().max().item() <= 2e-2
    assert (lse - c.lse).abs().max().item() <= 2e-3


@pytest.mark.gpu
def test_two_streams_give_the_same_bytes(A):
    """Calls that overlap on two streams do not share workspace; a repeated call is bit-identical."""
    a = Case("bf16", 8, 2, 128, 16, [24, 24], [900, 2000], "tree", 13)
    b = Case("e4m3", 8, 2, 128, 16, [2, 2], [3000, 2000], "tree", 14)
    want = []
    for c in (a, b):
        c.run(A, 6)
        want.append((c.o.clone(), c.lse.clone()))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip((a, b), streams):
            c.run(A, 6, stream=s)
    torch.cuda.synchronize()
    for c, (o, lse) in zip((a, b), want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d,page", [("bf16", 4, 128, 16), ("e5m2", 2, 64, 7), ("e4m3", 3, 128, 16), ("bf16", 20, 128, 16),
                                          ("bf16", 33, 64, 5), ("e4m3", 20, 128, 16), ("e5m2", 40, 64, 64)])
@pytest.mark.parametrize("num_splits", [2, 8, 9, 40])
def test_splits_joined_in_a_cluster_or_by_a_second_kernel(A, fmt, n, d, page, num_splits):
    """Up to eight splits that all fit at once are joined by their blocks; sequences of fewer splits, of one, of no
    tokens and of no rows among them, and a non-finite value that every row of a sequence sees."""
    c = Case(fmt, 4, 2, d, page, [n, n, 0, 1, n], [2600, n + 70, 0, 1, n + 700], "tree", 23)
    c.run(A, num_splits)
    o, lse = c.o.clone(), c.lse.clone()
    c.run(A, num_splits)
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert A.attn_get_device_status() == 0
    c.check()
    tok = 1300
    row = int(c.pt[0, tok // page]) * page + tok % page
    c.c[1].view(-1, 2, d)[row, 1, 5] = float("nan") if fmt == "bf16" else 0x7F
    c.run(A, num_splits)
    nan = torch.isnan(c.o)
    want = torch.zeros_like(nan)
    want[:n, 2:, 5] = True
    assert torch.equal(nan, want)
    assert torch.equal(c.o[~nan], o[~nan]) and torch.equal(c.lse, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("num_splits", [8, 20])
def test_streams_at_once_with_few_and_many_splits(A, num_splits):
    cases = [Case("bf16", 8, 2, 128, 16, [24, 24], [900, 2000], "tree", 13), Case("e4m3", 8, 2, 128, 16, [2, 2], [3000, 2000], "tree", 14),
             Case("e5m2", 8, 8, 64, 16, [24], [2500], "chain", 15)]
    want = []
    for c in cases:
        c.run(A, num_splits)
        want.append((c.o.clone(), c.lse.clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            c.run(A, num_splits, stream=s)
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cases, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
        c.check()
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,Hq", [("bf16", 1), ("e4m3", 17)])
def test_more_sequences_than_grid_rows_for_two_orders(A, fmt, Hq):
    """With two splits and more than half of 65535 sequences the splits of a sequence share a grid row; the second kernel
    joins them."""
    rs = np.random.RandomState(30)
    B = 33000
    lens = [int(x) for x in rs.randint(0, 20, B)]
    for b, l in ((0, 150), (1, 64), (2, 129), (B - 1, 150)):
        lens[b] = l
    c = Case(fmt, Hq, 1, 64, 16, [1] * B, lens, "chain", 31, dense=True)
    c.run(A, 2)
    assert A.attn_get_device_status() == 0
    if Hq > 1:  # every row and head of some of them
        some = [*range(4), *range(4, B - 4, 400), *range(B - 4, B)]
        c.q, c.o, c.lse, c.pt = c.q[some], c.o[some], c.lse[some], c.pt[some]
        c.n, c.lens, c.seen, c.T, c.cu = [1] * len(some), [c.lens[b] for b in some], [c.seen[b] for b in some], len(some), np.arange(len(some) + 1)
    c.check()


@pytest.mark.gpu
def test_calls_from_several_host_threads(A):
    """Threads with a stream and buffers each, through clusters, workspaces and both kernels, give the bytes of calls one
    after the other."""
    import threading
    cases = [(Case("bf16", 8, 2, 128, 16, [24, 24], [900, 2000], "tree", 13), 0), (Case("e4m3", 8, 2, 128, 16, [2, 2], [3000, 2000], "tree", 14), 20),
             (Case("e5m2", 8, 8, 64, 7, [24], [2500], "chain", 15), 8), (Case("bf16", 16, 8, 64, 16, [3] * 12, [40 * i + 3 for i in range(12)], "any", 16), 0)]
    want = []
    for c, splits in cases:
        c.run(A, splits)
        want.append((c.o.clone(), c.lse.clone()))
    torch.cuda.synchronize()
    failed = []

    def work(c, splits, o, lse):
        try:
            s = torch.cuda.Stream()
            for _ in range(30):
                with torch.cuda.stream(s):
                    c.o.fill_(7)
                c.run(A, splits, stream=s)
            s.synchronize()
            if not (torch.equal(c.o, o) and torch.equal(c.lse, lse)):
                failed.append("other bytes")
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(*c, *w)) for c, w in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and A.attn_get_device_status() == 0
    for c, _ in cases:
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("num_splits", [8, 20])
def test_two_graphs_replayed_at_once(A, num_splits):
    """Each captured call has a workspace of its own: replays on two streams give the bytes of calls one after the other."""
    cases = [Case("bf16", 8, 2, 128, 16, [24, 24], [900, 2000], "tree", 13), Case("bf16", 8, 2, 128, 16, [24, 24], [1900, 1000], "tree", 17),
             Case("e4m3", 8, 2, 64, 16, [3, 2], [3000, 2000], "tree", 14)]
    want, graphs, streams = [], [], []
    for c in cases:
        c.run(A, num_splits)
        want.append((c.o.clone(), c.lse.clone()))
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                c.run(A, num_splits)
        graphs.append(g)
        streams.append(s)
        c.o.fill_(7)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cases, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,Hq,Hkv,n,d", [("bf16", 600, 1, 2, 64), ("e4m3", 700, 1, 1, 128), ("e5m2", 900, 900, 1, 64), ("bf16", 1000, 500, 9, 64)])
def test_many_heads(A, fmt, Hq, Hkv, n, d):
    c = Case(fmt, Hq, Hkv, d, 16, [n, n], [n + 30, n + 200], "tree", 18)
    c.run(A)
    assert A.attn_get_device_status() == 0
    c.check()


BATCHES = {  # cached tokens of each sequence, and how many times wider than needed the page table is
    "equal": ([512] * 20, 1),
    "ragged": ([(i * 97) % 500 + 20 for i in range(18)] + [0, 22], 1),
    "one_long": ([20 + i % 3 for i in range(15)] + [6000], 1),
    "wide_table": ([64 * (i + 1) for i in range(10)], 12),
    "many": ([20 + (i * 37) % 300 for i in range(63)], 3),
    "all_empty": ([0] * 20, 30),
}


def widened(c, times):
    pt = np.full((c.B, c.width * times), 2**31 - 1, np.int32)
    pt[:, :c.width] = c.pt
    c.pt, c.width = pt, c.width * times
    c.dev["pt"] = torch.from_numpy(pt).to(DEV)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d", [("bf16", 2, 128), ("e4m3", 2, 64), ("bf16", 20, 64), ("e4m3", 20, 128)])
@pytest.mark.parametrize("batch", BATCHES)
def test_splits_chosen_by_the_lengths(A, fmt, n, d, batch):
    """Batches of fewer groups than the GPU holds blocks: the split size follows the lengths."""
    lens, times = BATCHES[batch]
    Hkv = 2 if batch == "many" else 8
    c = widened(Case(fmt, Hkv, Hkv, d, 16, [n] * len(lens), lens, "tree", 21), times)
    c.run(A)
    o, lse = c.o.clone(), c.lse.clone()
    c.run(A)
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d", [("bf16", 20, 128), ("bf16", 40, 64), ("e5m2", 40, 64)])
@pytest.mark.parametrize("batch", ["ragged", "one_long", "wide_table"])
def test_tiles_split_by_the_lengths(A, fmt, n, d, batch):
    lens, times = BATCHES[batch]
    lens = [x and max(x, n) for x in lens]
    c = widened(Case(fmt, 8, 8, d, 16, [n] * len(lens), lens, "tree", 24), times)
    c.run(A)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n,d,page", [("bf16", 20, 128, 7), ("bf16", 40, 64, 1), ("e4m3", 20, 128, 24), ("e5m2", 40, 64, 13)])
@pytest.mark.parametrize("batch", ["ragged", "one_long", "wide_table"])
def test_tiles_of_odd_pages_split_by_the_lengths(A, fmt, n, d, page, batch):
    """Page sizes that no box divides (rows are copied one by one, and there are no tensor maps)."""
    lens, times = BATCHES[batch]
    lens = [x and max(x, n) for x in lens]
    c = widened(Case(fmt, 8, 8, d, page, [n] * len(lens), lens, "tree", 25), times)
    c.run(A)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,page", [("bf16", 16), ("bf16", 5), ("e4m3", 64), ("e5m2", 7)])
@pytest.mark.parametrize("B,Hkv,times", [(4, 2, 1), (4, 2, 9000), (80, 1, 1), (80, 2, 1)])
def test_narrow_heads_whatever_the_table_holds(A, fmt, page, B, Hkv, times):
    """17 to 32 rows of 64 elements where 16-row products and where tiles are taken: small and very wide tables, more
    sequences than the lengths are looked at for."""
    rs = np.random.RandomState(5)
    lens = [int(x) for x in rs.randint(6, 200, B)]
    c = widened(Case(fmt, 4 * Hkv, Hkv, 64, page, [6] * B, lens, "any", 29), times)
    c.run(A)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("n,page,num_splits", [(5, 16, 0), (8, 7, 1), (7, 1, 3), (6, 64, 12), (8, 16, 8)])
def test_two_row_groups_of_narrow_heads(A, fmt, n, page, num_splits):
    """17 to 32 rows of 64 elements: ragged row counts whose second group is partly or wholly empty, rows that see
    nothing, a masked NaN."""
    c = Case(fmt, 8, 2, 64, page, [n, 1, n - 1, 0, n], [n + 900, 1, n + 60, 5, n], "any", 26)
    tok = c.lens[0] - n  # the first drafted token, which no row is to see
    c.seen[0][:, 0] = False
    m = c.mask.cpu().numpy().view(np.uint64)
    m[:n] &= ~np.uint64(1)
    c.mask = torch.from_numpy(m.view(np.int64)).to(DEV)
    for cache in c.c:
        cache.view(-1, 2, 64)[int(c.pt[0, tok // page]) * page + tok % page] = float("nan") if fmt == "bf16" else 0x7F
    c.run(A, num_splits)
    assert A.attn_get_device_status() == 0
    keep = c.values
    c.values = lambda: [np.nan_to_num(x, nan=0.0) for x in keep()]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,B,n,Hkv,d", [("bf16", 70, 2, 2, 128), ("e4m3", 300, 1, 2, 64), ("bf16", 70, 18, 1, 128), ("e5m2", 45, 18, 8, 128),
                                           ("bf16", 100, 1, 8, 128)])
@pytest.mark.parametrize("num_splits", [0, 3])
def test_more_groups_than_blocks_at_once(A, fmt, B, n, Hkv, d, num_splits):
    """Many sequences: last splits after all others, longest first (up to 256 sequences)."""
    rs = np.random.RandomState(27)
    lens = [int(x) for x in rs.randint(n, 400, B)]
    lens[3], lens[B - 1] = 0, 900
    c = Case(fmt, Hkv, Hkv, d, 16, [n] * B, lens, "tree", 28)
    c.run(A, num_splits)
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("bf16", 2), ("e4m3", 20)])
def test_replay_with_other_lengths(A, fmt, n):
    """The split size of a graph's call follows the lengths of each replay, a bad one among them."""
    full = [800, 300] * 8
    c = widened(Case(fmt, 8, 8, 64, 16, [n] * 16, full, "chain", 22, dense=True), 5)
    c.run(A)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(A)
    for lens in ([n] * 16, [800] + [n + 1] * 15, full, [n + 250] * 16):
        c.lens = lens
        c.dev["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        c.dev["lens"][3] = 10**9 if lens is full else lens[3]
        g.replay()
        bad = A.attn_get_device_status()
        assert bad == (A.ATTN_ERR_DEVICE_BAD_INDEX if lens is full else 0)
        c.lens = [0 if lens is full and b == 3 else x for b, x in enumerate(lens)]
        c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 20])
def test_captured_and_replayed(A, fmt, n):
    """A graph follows new queries, lengths and masks in the captured buffers."""
    c = Case(fmt, 8, 2, 128, 16, [n] * 3, [n + 500, n + 40, n + 900], "tree", 15, dense=True)
    c.run(A)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(A)
    c.q.copy_(torch.randn_like(c.q))
    c.dev["lens"].sub_(7)
    c.mask.bitwise_or_(1)  # every node sees the first one too
    c.lens = [x - 7 for x in c.lens]
    for s in c.seen:
        s[:, 0] = True
    c.o.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert A.attn_get_device_status() == 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("n", [3, 24])
def test_step_rotate_write_attend_read(A, fmt, n):
    """A serving step as its calls: q and k rotated at the nodes' depths out of one projection, keys
    and values written behind the context, the tree attended, the drafted rows read back."""
    Hq, Hkv, d, page = 8, 2, 128, 16
    c = Case(fmt, Hq, Hkv, d, page, [n, n - 1], [n + 50, 200 + n], "tree", 16)
    T, W = c.T, (Hq + 2 * Hkv) * d
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((T, W), generator=g).bfloat16().to(DEV)
    freqs, amp = A.attn_rope_freqs(d)
    inv = torch.tensor(freqs, dtype=torch.float64, device=DEV)
    depth = np.zeros(T, np.int32)
    for b, m in enumerate(c.n):
        depth[c.cu[b]:c.cu[b] + m] = c.lens[b] - m + c.seen[b].sum(1) - 1
    pos = torch.from_numpy(depth).to(DEV)
    k, v = qkv[:, Hq * d:(Hq + Hkv) * d], qkv[:, (Hq + Hkv) * d:]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A.attn_rope(qkv, None, c.q, None, pos, inv, T, Hq, 0, d, 0, d, W, 0, Hq * d, 0, amplitude=amp)
        A.attn_kv_write_paged(k, v, W, W, c.c[0], c.c[1], c.dev["pt"], c.dev["lens"], c.dev["cu"], page, T, c.B, Hkv, d, c.width, c.num,
                              fmt, *c.ds, positions=pos, inv_freq=inv, rot_dim=d, amplitude=amp)
        c.run(A)
        kr, vr = (torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        A.attn_kv_read_paged(c.c[0], c.c[1], kr, vr, Hkv * d, Hkv * d, c.dev["pt"], c.dev["lens"], c.dev["cu"], page, T, c.B, Hkv, d,
                             c.width, c.num, fmt, *c.ds)
    s.synchronize()
    assert A.attn_get_device_status() == 0
    c.check()  # on the cache and the queries as the calls left them
    m = sum(c.n)
    # the read-back rows are the projection's: one rounding to the cache's format, one to bf16
    step = {"bf16": 0.0, "e4m3": 2.0**-4, "e5m2": 2.0**-3}[fmt]
    floor = 0.0 if fmt == "bf16" else c.ds[1] * {"e4m3": 2.0**-10, "e5m2": 2.0**-17}[fmt]
    x = v[:m].double().reshape(m, Hkv, d)
    assert ((vr[:m].double() - x).abs() <= x.abs() * (step + 2.0**-8 * (step > 0)) * 1.01 + floor).all()
    assert (vr[m:] == 7).all() and (kr[m:] == 7).all()
    # rotation keeps each pair's length: keys too, up to the roundings of both members
    z = k[:m].double().reshape(m, Hkv, d)
    before = (z[..., :64] ** 2 + z[..., 64:] ** 2).sqrt()
    after = (kr[:m, :, :64].double() ** 2 + kr[:m, :, 64:].double() ** 2).sqrt()
    assert ((after - before).abs() <= before * (step + 2.0**-7) * 1.5 + 2 * floor).all()
