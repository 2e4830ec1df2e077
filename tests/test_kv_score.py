"""attn_kv_score_paged: refusals on the CPU; on the GPU every slot against 64-bit arithmetic with a bound that counts the
roundings, untouched slots bit for bit, bad lengths, offsets and pages recorded."""
import math

import numpy as np
import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")
DEV = "cuda:0"
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def A():
    ensure_built()
    import exact_softmax_attention_gb300 as mod
    return mod


# ------------------------------------------------------------------------------------- CPU

def status(A, **kw):
    a = dict(q=0x1000, lse=0x2000, k_cache=0x3000, score=0x4000, page_table=0x5000, seqlens=0x6000, cu_seqlens=None, page_size=16, T=0, B=1,
             max_q=1, Hq=4, Hkv=2, d=128, max_pages_per_seq=4, num_pages=8, scale=0.1, decay=1.0, kv_format="e4m3", k_descale=0.5)
    a.update(kw)
    return A.attn_kv_score_paged(**a, stream=0, raise_on_error=False)


def test_refusals(A):
    null, shape, align, arg = A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    assert status(A) == A.ATTN_OK and status(A, B=0) == A.ATTN_OK and status(A, decay=0.0, scale=-1.0) == A.ATTN_OK
    for name in ("q", "lse", "k_cache", "score", "page_table", "seqlens"):
        assert status(A, **{name: None}) == null
    for bad in (dict(T=-1), dict(B=-1), dict(B=65536), dict(max_q=0), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=65536 * 2, Hkv=65536),
                dict(d=96), dict(d=256), dict(page_size=0), dict(max_pages_per_seq=0), dict(num_pages=0), dict(num_pages=1 << 27),
                dict(max_pages_per_seq=1 << 26), dict(T=5, B=2, max_q=9), dict(T=5, B=0), dict(T=6, B=2, max_q=2), dict(T=1 << 30, max_q=1 << 30),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert status(A, **bad) == shape, bad
    for bad in (dict(kv_format=3), dict(kv_format=-1), dict(k_descale=float("nan")), dict(decay=float("inf")), dict(decay=float("nan")),
                dict(scale=1e30, k_descale=1e30)):
        assert status(A, **bad) == arg, bad
    for bad in (dict(q=0x1008), dict(k_cache=0x3008), dict(lse=0x2002), dict(score=0x4001), dict(page_table=0x5002), dict(seqlens=0x6001),
                dict(cu_seqlens=0x7002)):
        assert status(A, **bad) == align, bad


# ------------------------------------------------------------------------------------- GPU

class Problem:
    """Sequences of `lens` cached tokens, the last n of which are queries; slots that no token holds are NaN keys."""

    def __init__(self, n, lens, Hq, Hkv, d, page, fmt, seed=0, tail=2, dense=False, q_size=2.0, scale=None):
        rs = np.random.RandomState(seed + d + page + len(n))
        self.n, self.lens, self.B = np.array(n), np.array(lens), len(n)
        self.Hq, self.Hkv, self.d, self.page, self.fmt, self.G = Hq, Hkv, d, page, fmt, Hq // Hkv
        pages = -(-self.lens // page)
        self.num, self.width = int(pages.sum()) + 2, int(max(1, pages.max())) + 1
        perm, self.pt, at = rs.permutation(self.num), np.full((self.B, self.width), 2**31 - 1, np.int32), 0
        for b, c in enumerate(pages):
            self.pt[b, :c] = perm[at:at + c]
            at += c
        self.T = int(self.n.sum()) + (0 if dense else tail)
        self.cu = None if dense else torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.q = (torch.randn((self.T, Hq, d), generator=g, device=DEV) * q_size).bfloat16()
        k = torch.randn((self.num, page, Hkv, d), generator=g, device=DEV)
        self.kds = 1.0 if fmt == "bf16" else 0.02
        held = torch.zeros((self.num, page), dtype=torch.bool, device=DEV)
        for b in range(self.B):
            pg, sl = self.places(b)
            held[pg, sl] = True
        if fmt == "bf16":
            self.kc = k.bfloat16()
            self.kc[~held] = float("nan")
        else:
            self.kc = (k / self.kds).clamp(-200, 200).to(F8[fmt]).view(torch.uint8)
            self.kc[~held] = 0x7F
        self.held = held
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.score = torch.rand((self.num, Hkv, page), generator=g, device=DEV) * 3
        self.ptd, self.lend = torch.from_numpy(self.pt).to(DEV), torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        self.max_q = int(max(1, self.n.max()))
        self.lse = torch.full((self.T, Hq), 7.0, device=DEV)
        at = 0
        for b in range(self.B):
            if self.n[b]:
                self.lse[at:at + self.n[b]] = self.logits(b).logsumexp(-1).float()
            at += self.n[b]

    def places(self, b):
        t = np.arange(self.lens[b])
        return torch.from_numpy(self.pt[b, t // self.page].astype(np.int64)).to(DEV), torch.from_numpy(t % self.page).to(DEV)

    def keys(self, b):
        """[tokens, Hkv, d] in 64 bits"""
        pg, sl = self.places(b)
        k = self.kc[pg, sl]
        return k.double() if self.fmt == "bf16" else k.view(F8[self.fmt]).double() * float(np.float32(self.kds))

    def logits(self, b, absolute=False):
        """[n, Hq, tokens] in 64 bits, -inf where masked"""
        at = int(self.n[:b].sum())
        q, k = self.q[at:at + self.n[b]].double(), self.keys(b)
        if absolute:
            q, k = q.abs(), k.abs()
        s = torch.einsum("nhgd,thd->nhgt", q.view(-1, self.Hkv, self.G, self.d), k).reshape(self.n[b], self.Hq, -1)
        s = s * (abs(self.scale) if absolute else self.scale)
        t, ctx = torch.arange(int(self.lens[b]), device=DEV), int(self.lens[b] - self.n[b])
        return s.masked_fill((t[None] > ctx + torch.arange(int(self.n[b]), device=DEV)[:, None])[:, None], 0.0 if absolute else float("-inf"))

    def run(self, A, decay=1.0, **kw):
        A.attn_kv_score_paged(self.q, self.lse, self.kc, self.score, self.ptd, self.lend, self.cu, self.page, self.T, self.B, self.max_q, self.Hq,
                              self.Hkv, self.d, self.width, self.num, self.scale, decay, self.fmt, self.kds, **kw)

    def check(self, before, decay, skip=()):
        touched = torch.zeros((self.num, self.page), dtype=torch.bool, device=DEV)
        worst, at = 0.0, 0
        for b in range(self.B):
            n, L = int(self.n[b]), int(self.lens[b])
            lse = self.lse[at:at + n].double()
            at += n
            if n == 0 or b in skip:
                continue
            pg, sl = self.places(b)
            touched[pg, sl] = True
            s, size = self.logits(b), self.logits(b, True)
            seen = lse > -math.inf
            p = torch.where(seen[..., None], (s - torch.where(seen, lse, 0.0)[..., None]).exp(), 0.0)
            # the product: d fp32 additions of |q k| (2^-23 each, for units that truncate), factor and difference in fp32, ex2 within
            # 2^-21; two 8-bit parts of q leave 2^-17 of the row's largest element times |k|
            e = size * self.d * 2.0**-23 + (s.abs().nan_to_num(posinf=0.0) + torch.where(seen, lse.abs(), 0.0)[..., None]) * 4 * 2.0**-24 + 2.0**-21
            if self.fmt != "bf16" and self.max_q * self.G > 24:
                top = self.q[at - n:at].double().abs().amax(-1).view(n, self.Hkv, self.G, 1)
                e = e + (top * self.keys(b).abs().sum(-1).T[None, :, None]).reshape(n, self.Hq, L) * abs(self.scale) * 2.0**-17
            group = lambda x: x.view(n, self.Hkv, self.G, L).sum((0, 2)).T
            new = group(p)
            # the sum: no term passes more than n G additions; the old value one product and one sum
            tol = group(p * torch.expm1(e)) + new * (n * self.G + 4) * 2.0**-24 + 1e-36
            old = before[pg, :, sl].double()
            old[L - n:] = 0  # the rows' own tokens are new
            ref = new + (decay * old if decay else 0)
            tol = tol + (ref.abs() + (abs(decay) * old if decay else 0)) * 2.0**-23
            got = self.score[pg, :, sl].double()
            bad = (got - ref).abs() > tol
            assert not bad.any(), (b, int(bad.sum()), ((got - ref).abs() / tol).max().item())
            worst = max(worst, ((got - ref).abs() / tol).max().item())
        # slots behind the sequences, of other pages and of sequences without rows are as they were
        keep = ~touched[:, None, :].expand_as(self.score)
        assert torch.equal(self.score[keep], before[keep])
        return worst


FEW = [  # rows, lengths, Hq, Hkv, d, page, dense
    ([1], [1], 1, 1, 64, 1, True),
    ([1] * 5, [1, 2, 17, 300, 1000], 8, 2, 128, 16, True),
    ([1] * 70, list(range(3, 73)), 4, 4, 64, 7, True),
    ([3, 0, 1, 4], [3, 50, 8, 900], 12, 3, 64, 5, False),
    ([2, 1], [40, 2000], 16, 2, 128, 64, False),          # 16 rows
    ([1, 1], [555, 1], 45, 9, 128, 16, True),             # more heads than warps of a block
    ([1], [130], 20, 20, 64, 100, True),
    ([16, 5], [16, 70], 5, 5, 128, 3, False),
    ([1], [20000], 3, 1, 128, 16, True),
    ([5, 3, 0, 4], [700, 30, 9, 1100], 8, 2, 128, 16, False),  # 20 and
    ([8, 1], [600, 3000], 8, 2, 64, 7, False),                 # 32 rows
    ([1] * 40, [3000 - 70 * i for i in range(40)], 16, 8, 128, 16, True),  # equal runs over ragged lengths
    ([1] * 300, [100 + 7 * i for i in range(300)], 12, 12, 64, 16, True),  # more sequences than threads, two groups of heads
]
MANY = [
    ([33], [33], 1, 1, 64, 1, True),
    ([17], [17], 2, 1, 64, 1, True),
    ([32, 0, 5, 31], [400, 9, 700, 31], 8, 2, 128, 16, False),
    ([33] * 3, [33, 256, 1025], 3, 1, 64, 7, True),       # a group that does not divide 128
    ([32] * 4, [3000, 100, 257, 513], 16, 4, 128, 64, True),  # 128 rows
    ([300, 1, 129, 64], [300, 1, 129, 64], 8, 2, 128, 16, False),  # whole prompts
    ([700, 40], [700, 1000], 8, 1, 64, 16, False),        # units split between the blocks
    ([1500], [1800], 8, 1, 128, 5, True),
    ([1000], [1000], 1, 1, 128, 256, True),
    ([40, 300], [300, 300], 200, 1, 64, 16, False),       # more heads of a kv head than a block of rows
    ([9, 50], [300, 260], 100, 1, 128, 16, False),        # one query per block
    ([400, 7], [600, 90], 10, 2, 64, 32, False),          # 25 queries per block
    ([600], [1100], 21, 3, 128, 128, True),
    ([32] * 12, [600 + 400 * i for i in range(12)], 16, 8, 128, 16, True),  # many units of 512 tokens and less for each block
    ([32] * 12, [600 + 400 * i for i in range(12)], 16, 8, 64, 7, True),
    ([20] * 500, [20 + i % 7 for i in range(500)], 1, 1, 64, 16, True),  # more sequences than a block's threads
]


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens,Hq,Hkv,d,page,dense", FEW + MANY)
@pytest.mark.parametrize("fmt,decay", [("bf16", 1.0), ("e4m3", 0.0), ("e5m2", 0.9), ("bf16", 0.0)])
def test_against_64_bits(A, n, lens, Hq, Hkv, d, page, dense, fmt, decay):
    p = Problem(n, lens, Hq, Hkv, d, page, fmt, dense=dense)
    first = p.score.clone()
    for b in np.flatnonzero(p.n):  # sums of new tokens, and without decay all, are not read
        pg, sl = p.places(b)
        from_ = 0 if decay == 0.0 else p.lens[b] - p.n[b]
        p.score[pg[from_:], :, sl[from_:]] = float("nan")
    before = p.score.clone()
    p.run(A, decay)
    assert A.attn_get_device_status() == 0
    p.check(before, decay)
    again, p.score = p.score, first
    p.run(A, decay)
    assert torch.equal(again, p.score)  # the same bytes


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [2, 4, 6, 8, 12, 24])
@pytest.mark.parametrize("d,fmt", [(64, "bf16"), (64, "e4m3"), (128, "bf16"), (128, "e5m2")])
def test_heads_of_a_block(A, Hkv, d, fmt):
    """One to 24 rows per kv head over numbers of heads that blocks take whole, in parts or a few at a time; short batches and many sequences."""
    for G, n in ((1, 1), (4, 1), (2, 8), (3, 8)):
        for B, length in ((1, 100), (50, 900)):
            p = Problem([n] * B, [n + (length * (i + 1)) // B for i in range(B)], G * Hkv, Hkv, d, 16, fmt, seed=9, dense=True)
            before = p.score.clone()
            p.run(A, 0.5)
            p.check(before, 0.5)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens,Hq,Hkv", [([1] * 3, [5, 40, 700], 8, 2), ([40, 20], [300, 200], 8, 2)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
def test_magnitudes_and_scales(A, n, lens, Hq, Hkv, fmt):
    """q far above and below the range of f16, a negative scale, sharp softmax."""
    for size, scale in ((1e30, 1e-31), (1e-30, 1e29), (2.0, -0.1), (6.0, 0.3), (2.0, 0.0)):
        p = Problem(n, lens, Hq, Hkv, 128, 16, fmt, seed=3, q_size=size, scale=scale)
        before = p.score.clone()
        p.run(A)
        assert A.attn_get_device_status() == 0
        p.check(before, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1, 1], [50, 300]), ([40, 33], [300, 200])])
def test_rows_that_saw_nothing_and_nan(A, n, lens):
    """Heads of lse = -inf add nothing; a NaN in q or K reaches the tokens that it belongs to only."""
    p = Problem(n, lens, 8, 2, 64, 16, "bf16", seed=4)
    p.lse[0, 1] = p.lse[n[0], 5] = -math.inf
    before = p.score.clone()
    p.run(A)
    p.check(before, 1.0)
    pg, sl = p.places(1)
    p.kc[pg[30], sl[30], 1, 7] = float("nan")
    p.q[n[0], 0, 3] = float("inf")  # kv head 0 of sequence 1
    p.score.copy_(before)
    p.run(A)
    got = p.score[pg, :, sl]
    first = lens[1] - n[1] + 1  # tokens that the row sees
    assert torch.isnan(got[30, 1]) and torch.isfinite(got[:30, 1]).all() and torch.isfinite(got[31:, 1]).all()
    odd = ~torch.isfinite(got[:, 0])
    assert not odd[first:].any()
    pg, sl = p.places(0)
    assert torch.isfinite(p.score[pg, :, sl]).all() and A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1, 1], [50, 300]), ([40, 33], [300, 200])])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.1, -0.1, 1e-15, 1e15, 1e-25, 1e25])
def test_lse_far_out(A, n, lens, fmt, scale):
    """An LSE far above every score gives weight 0, one far below weight infinity, NaN gives NaN to the tokens that its row sees."""
    p = Problem(n, lens, 8, 2, 128, 16, fmt, seed=6, q_size=2.0 / max(1.0, abs(scale)), scale=scale)
    first = lens[1] - n[1]  # the last token that the first row of sequence 1 sees
    kept = p.lse.clone()
    before, results = p.score.clone(), []
    for value in (-math.inf, math.inf, 3e38, 1e9):
        p.lse.copy_(kept)
        p.lse[:, 0::4] = value  # a query head of each kv head
        p.score.copy_(before)
        p.run(A)
        results.append(p.score.clone())
    assert all(torch.equal(results[0], x) for x in results[1:])  # as heads that saw nothing
    for value, wrong in ((-3e38, torch.isposinf), (-1e9, torch.isposinf), (math.nan, torch.isnan)):
        p.lse.copy_(kept)
        p.lse[n[0], 3] = value  # kv head 0
        p.score.zero_()
        p.run(A)
        pg, sl = p.places(1)
        got = p.score[pg, :, sl]
        assert wrong(got[:first + 1, 0]).all() and torch.isfinite(got[first + 1:, 0]).all() and torch.isfinite(got[:, 1]).all()
        pg, sl = p.places(0)
        assert torch.isfinite(p.score[pg, :, sl]).all()
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1, 1, 1], [50, 300, 20]), ([40, 33, 5], [300, 200, 20]), ([500, 33, 5], [600, 200, 20])])
def test_bad_lengths_pages_and_offsets(A, n, lens):
    bad = A.ATTN_ERR_DEVICE_BAD_INDEX
    make = lambda: Problem(n, lens, 8, 2, 64, 16, "bf16", seed=5)
    for value in (n[1] - 1, -3, make().width * 16 + 1):  # below the rows, negative, above the table
        p = make()
        before = p.score.clone()
        p.lend[1] = value
        p.run(A)
        assert A.attn_get_device_status() == bad
        p.check(before, 1.0, skip=(1,))
    for at, value in ((3, 2**30), (1, n[0] + n[1] + 1), (2, n[0] - 1)):  # the last one passes T; others decrease behind it
        p = make()
        before = p.score.clone()
        p.cu[at] = value
        p.run(A)
        assert A.attn_get_device_status() == bad
        if at == 3:
            p.check(before, 1.0, skip=(2,))
    for value in (-1, p.num):  # a page out of range: its slots are nobody's
        p = make()
        before = p.score.clone()
        real = p.pt[1, 0]
        p.ptd[1, 0] = value
        p.run(A)
        assert A.attn_get_device_status() == bad
        assert torch.equal(p.score[real], before[real])
        p.score[real] = 0
        q = make()
        q.run(A)
        q.score[real] = 0
        assert torch.equal(p.score, q.score)


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1] * 4, [5, 300, 1000, 64]), ([64, 200, 30, 1], [300, 1000, 64, 70])])
def test_streams_and_graph(A, n, lens):
    """Two captured calls replayed at once on two streams, then on new lengths; eager calls between."""
    ps = [Problem(n, lens, 8, 2, 128, 16, fmt, seed=6) for fmt in ("bf16", "e4m3")]
    start = [p.score.clone() for p in ps]
    want = []
    for p in ps:
        p.run(A)
        want.append(p.score.clone())
    graphs, streams = [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(A)
        graphs.append(g)
    for _ in range(3):
        for p, x in zip(ps, start):
            p.score.copy_(x)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for p, w in zip(ps, want):
            assert torch.equal(p.score, w)
    p = ps[0]
    p.lens[2] -= 5  # one page fewer tokens in use: the queries are those of earlier tokens
    p.lend.copy_(torch.from_numpy(p.lens.astype(np.int32)))
    p.score.copy_(start[0])
    graphs[0].replay()
    torch.cuda.synchronize()
    p.check(start[0], 1.0)
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,n", [("bf16", 1), ("e4m3", 1), ("bf16", 20), ("e5m2", 20)])
def test_cache_offsets_beyond_32_bits(A, fmt, n):
    """Tokens on the last pages of a cache of more than 2^31 elements against the same tokens in a small one."""
    Hkv, d, page = 8, 128, 16
    num = 2**31 // (page * Hkv * d) + 9
    p = Problem([n, n], [30, 45], 16, Hkv, d, page, fmt, seed=7)
    before = p.score.clone()
    big = torch.empty((num, page, Hkv, d), dtype=p.kc.dtype, device=DEV)
    score = torch.zeros((num, Hkv, page), device=DEV)
    far = num - 1 - torch.arange(p.num, device=DEV)
    big[far], score[far] = p.kc, p.score
    pt = torch.where((p.ptd >= 0) & (p.ptd < p.num), num - 1 - p.ptd, p.ptd)
    A.attn_kv_score_paged(p.q, p.lse, big, score, pt, p.lend, p.cu, page, p.T, p.B, p.max_q, 16, Hkv, d, p.width, num, p.scale, 1.0, fmt, p.kds)
    p.run(A)
    assert torch.equal(score[far], p.score) and A.attn_get_device_status() == 0
    p.check(before, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_weights_of_a_decode_and_a_prefill_add_up(A, fmt):
    """With the LSE that the library's attention returns, each row's weights add up to one."""
    B, Hq, Hkv, d, page = 3, 8, 2, 128, 16
    p = Problem([1] * B, [40, 900, 333], Hq, Hkv, d, page, fmt, seed=8, dense=True)
    o, vc = torch.empty_like(p.q), torch.nan_to_num(p.kc) if fmt == "bf16" else p.kc
    if fmt == "bf16":
        A.attn_decode_paged(p.q, p.kc, vc, p.ptd, p.lend, page, o, p.lse, None, B, Hq, Hkv, d, p.width, p.num, p.scale)
    else:
        A.attn_decode_paged_fp8(p.q, p.kc, vc, p.ptd, p.lend, page, o, p.lse, None, B, Hq, Hkv, d, p.width, p.num, p.scale, 0, fmt, p.kds, 1.0)
    p.run(A, 0.0)
    for b in range(B):
        pg, sl = p.places(b)
        total = p.score[pg, :, sl].double().sum(0)
        # the LSE is within 2e-3 of the exact one (the library's bar), which the weights' sum shows as a factor
        assert (total / (Hq // Hkv) - 1).abs().max() <= 2.1e-3
    if fmt == "bf16":
        n = 300
        k = torch.randn((n, Hkv, d), device=DEV).bfloat16()
        q = torch.randn((n, Hq, d), device=DEV).bfloat16()
        o, lse = torch.empty_like(q), torch.empty((n, Hq), device=DEV)
        A.attn_fwd(q, k, k, o, lse, 1, Hq, Hkv, n, n, d, p.scale, 1)
        pages = -(-n // page)
        kc = torch.zeros((pages, page, Hkv, d), dtype=torch.bfloat16, device=DEV)
        kc.view(-1, Hkv, d)[:n] = k
        score = torch.empty((pages, Hkv, page), device=DEV)
        A.attn_kv_score_paged(q, lse, kc, score, torch.arange(pages, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV),
                              None, page, n, 1, n, Hq, Hkv, d, pages, pages, p.scale, 0.0)
        total = score.permute(0, 2, 1).reshape(-1, Hkv)[:n].double().sum(0)
        assert (total / (n * Hq // Hkv) - 1).abs().max() <= 2.1e-3
    assert A.attn_get_device_status() == 0


# ------------------------------------------------------------------------------------- CPU: the host's cache of answers

def test_resident_blocks_by_device(tmp_path):
    """How many blocks an SM holds is known per device, and an answer that could not be had is asked for again: the function itself, from the
    source, with the CUDA calls replaced."""
    import ctypes
    import os
    import re
    import subprocess

    from helpers import ROOT
    with open(os.path.join(ROOT, "exact_softmax_attention_gb300", "csrc", "attn_score.cu")) as f:
        function = re.search(r"template <typename Kernel>\nint resident_blocks\(.*?\n}\n", f.read(), flags=re.S).group(0)
    src = tmp_path / "resident.cpp"
    src.write_text("""#include <atomic>
typedef int cudaError_t;
constexpr int cudaSuccess = 0, kMaxAttrDevices = 64, kRowWarps = 8;
static int answer, pending;
static int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, int, int, int) {
    if (answer < 0) return pending = 1;
    *n = answer;
    return 0;
}
static int cudaGetLastError() { const int e = pending; pending = 0; return e; }
""" + function + """
static std::atomic<int> known[kMaxAttrDevices][kRowWarps + 1];
extern "C" int ask(int device, int threads, int a) { answer = a; return resident_blocks(0, device, threads, known); }
extern "C" int left() { return pending; }
""")
    lib = tmp_path / "resident.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    c = ctypes.CDLL(str(lib))
    assert c.ask(0, 64, 5) == 5 and c.ask(0, 64, 9) == 5  # kept
    assert c.ask(0, 96, 4) == 4 and c.ask(1, 64, 7) == 7  # of other blocks, on another device
    assert c.ask(2, 64, -1) == 1 and c.left() == 0        # no answer: one block for this call, and no error left behind
    assert c.ask(2, 64, 6) == 6
    assert c.ask(64, 64, 3) == 3 and c.ask(64, 64, 2) == 2 and c.ask(-1, 64, 8) == 8


# ------------------------------------------------------------------------------------- GPU: precision, refusals and strays, closer

@pytest.mark.gpu
@pytest.mark.parametrize("d,G,n", [(64, 4, 8), (64, 4, 7), (64, 2, 13), (64, 1, 25), (64, 3, 8), (64, 4, 1), (128, 4, 6), (128, 2, 9), (128, 8, 1)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("B,length", [(3, 200), (40, 1500)])
def test_8_bit_keys_with_few_rows_are_exact(A, d, G, n, fmt, B, length):
    """Up to 32 rows per kv head of 64, 24 of 128, codes are widened exactly and q keeps elements down to 2^-29 of the row's largest. One element
    of each row is 2^11 to 2^14, the others are a few, and it meets keys of zero, so what a coarser q loses is far outside the bound."""
    Hkv = 2
    p = Problem([n] * B, [n + (length * (i + 1)) // B for i in range(B)], G * Hkv, Hkv, d, 16, fmt, seed=12, dense=True)
    big = 2.0 ** torch.randint(11, 15, (p.T, G * Hkv), device=DEV)
    p.q[..., 5] = big.bfloat16()
    zeroed = p.kc[..., 5]
    zeroed[p.held] = 0
    at = 0
    for b in range(B):
        p.lse[at:at + n] = p.logits(b).logsumexp(-1).float()
        at += n
    before = p.score.clone()
    p.run(A, 0.5)
    assert A.attn_get_device_status() == 0
    p.max_q = 0  # (the check's allowance for q in two parts is for more rows)
    p.check(before, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1, 1, 1], [50, 300, 20]), ([40, 33, 5], [300, 200, 90]), ([500, 33, 5], [600, 200, 90]), ([3, 2, 1], [30, 50, 9])])
@pytest.mark.parametrize("at,value", [(3, "far"), (3, "past"), (1, "both"), (2, "back"), (1, "negative"), (0, "skip"), (0, "negative")])
def test_bad_offsets_touch_nothing_else(A, n, lens, at, value):
    """Sequences whose offsets are out of range keep their slots bit for bit; those whose offsets stay valid get the sums of the rows that
    they then own."""
    import copy
    p = Problem(n, lens, 8, 2, 64, 16, "bf16", seed=5)
    before = p.score.clone()
    p.cu[at] = {"far": 2**30, "past": p.T + 1, "both": n[0] + n[1] + 1, "back": n[0] - 1, "negative": -2, "skip": 1}[value]
    cu = p.cu.tolist()
    p.run(A, 0.5)
    refused = 0
    expected = before.clone()
    for b in range(3):
        c0, c1 = cu[b:b + 2]
        rows = c1 - c0
        if rows == 0:
            continue
        if c0 < 0 or rows < 0 or c1 > p.T or rows > p.max_q or lens[b] < rows:
            refused += 1
            continue
        one = copy.copy(p)
        one.n, one.lens, one.B, one.pt = np.array([rows]), np.array(lens[b:b + 1]), 1, p.pt[b:b + 1]
        one.q, one.lse = p.q[c0:c1], p.lse[c0:c1]
        pg, sl = p.places(b)
        one.score = before.clone()
        one.score[pg, :, sl] = expected[pg, :, sl] = p.score[pg, :, sl]
        one.check(before, 0.5)
    assert torch.equal(p.score, expected)
    assert A.attn_get_device_status() == (A.ATTN_ERR_DEVICE_BAD_INDEX if refused else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1, 1], [50, 300]), ([6, 2], [50, 300]), ([40, 33], [300, 200]), ([300, 200], [300, 900])])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
def test_nan_reaches_what_sees_it_and_nothing_else(A, n, lens, fmt):
    """A NaN in a row of q makes the sums of exactly those tokens NaN that the row sees, of its kv head; all others are the same bytes as without
    it. So are all but one for a NaN in a key."""
    p = Problem(n, lens, 8, 2, 64, 16, fmt, seed=14)
    start = p.score.clone()
    p.run(A)
    clean = p.score.clone()
    row, head, i = n[0] + n[1] // 2, 6, n[1] // 2  # a query head of kv head 1, in the middle of sequence 1
    q = p.q.clone()
    p.q[row, head, 9] = math.nan
    p.score.copy_(start)
    p.run(A)
    pg, sl = p.places(1)
    seen = lens[1] - n[1] + i + 1
    wrong = torch.zeros_like(clean, dtype=torch.bool)
    wrong[pg[:seen], 1, sl[:seen]] = True
    assert torch.isnan(p.score[wrong]).all() and torch.equal(p.score[~wrong], clean[~wrong])
    p.q.copy_(q)
    token = min(37, lens[1] - 1)
    p.kc[pg[token], sl[token], 0, 3] = math.nan if fmt == "bf16" else 0x7F
    p.score.copy_(start)
    p.run(A)
    wrong.zero_()
    wrong[pg[token], 0, sl[token]] = True
    assert torch.equal(p.score[~wrong], clean[~wrong])
    assert A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,lens", [([1], [2000]), ([1] * 9, [5, 40, 700, 1, 300, 20, 90, 1100, 64]), ([40, 20], [300, 200]), ([700], [700])])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [131072, 2**20])
def test_short_sequences_in_a_wide_table(A, n, lens, fmt, tokens):
    """A page table for the longest context that a server allows, and sequences far below it."""
    p = Problem(n, lens, 8, 2, 128, 16, fmt, seed=15)
    p.ptd = torch.nn.functional.pad(p.ptd, (0, tokens // 16 - p.width), value=-1).contiguous()
    p.width = tokens // 16
    before = p.score.clone()
    p.run(A, 0.5)
    assert A.attn_get_device_status() == 0
    p.check(before, 0.5)


@pytest.mark.gpu
def test_calls_from_several_host_threads(A):
    """Calls of different sizes at once, each thread on a stream of its own: the same bytes as one after the other."""
    from concurrent.futures import ThreadPoolExecutor
    ps = [Problem(n, lens, 8, 2, d, page, fmt, seed=16) for d, page, fmt in ((64, 16, "bf16"), (128, 7, "e4m3"), (128, 16, "bf16"))
          for n, lens in (([1] * 5, [40, 900, 333, 1, 2000]), ([40, 20], [300, 200]), ([300], [800]))]
    start = [p.score.clone() for p in ps]
    for p in ps:
        p.run(A)
    want = [p.score.clone() for p in ps]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                ps[i].score.copy_(start[i])
                ps[i].run(A)
        s.synchronize()

    torch.cuda.synchronize()
    with ThreadPoolExecutor(len(ps)) as pool:
        list(pool.map(work, range(len(ps))))
    for p, w in zip(ps, want):
        assert torch.equal(p.score, w)
    assert A.attn_get_device_status() == 0
