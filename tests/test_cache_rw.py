"""attn_kv_write_paged and attn_kv_read_paged: refusals on the CPU; on the GPU every cache slot
against 64-bit arithmetic, untouched slots bit for bit, and bad lengths and pages recorded."""
import math

import numpy as np
import pytest

from helpers import ensure_built
from test_rope import reference as rope_reference

torch = pytest.importorskip("torch")
DEV = "cuda:0"
F8 = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}  # mantissa bits, least exponent, largest value


@pytest.fixture(scope="module")
def A():
    ensure_built()
    import exact_softmax_attention_gb300 as mod
    return mod


# ------------------------------------------------------------------------------------- CPU

def status(A, op, **kw):
    a = dict(k=0x1000, v=0x2000, k_stride=256, v_stride=256, k_cache=0x3000, v_cache=0x4000, page_table=0x5000, seqlens=0x6000,
             cu_seqlens=None, page_size=16, T=0, B=1, Hkv=2, d=128, max_pages_per_seq=4, num_pages=8, kv_format="e4m3", k_descale=0.5,
             v_descale=2.0)
    if op == "write":
        a.update(positions=None, inv_freq=None, rot_begin=0, rot_dim=0, interleaved=0, amplitude=1.0)
    a.update(kw)
    f = A.attn_kv_write_paged if op == "write" else A.attn_kv_read_paged
    return f(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("op", ["write", "read"])
def test_refusals(A, op):
    null, shape, align, arg = A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    assert status(A, op) == A.ATTN_OK and status(A, op, B=0) == A.ATTN_OK
    for name in ("k", "v", "k_cache", "v_cache", "page_table", "seqlens"):
        assert status(A, op, **{name: None}) == null
    for bad in (dict(T=-1), dict(B=-1), dict(Hkv=0), dict(Hkv=65536), dict(d=0), dict(d=72), dict(d=272), dict(page_size=0),
                dict(max_pages_per_seq=0), dict(num_pages=0), dict(num_pages=1 << 27, page_size=16),
                dict(max_pages_per_seq=1 << 27, page_size=16), dict(T=5, B=2), dict(T=5, B=0), dict(k_stride=260), dict(v_stride=-8)):
        assert status(A, op, **bad) == shape, bad
    if op == "read":
        assert status(A, op, k_stride=248) == shape and status(A, op, v_stride=0) == shape
    else:
        assert status(A, op, k_stride=0) == A.ATTN_OK  # one row repeated
    for bad in (dict(kv_format=3), dict(kv_format=-1), dict(k_descale=0.0), dict(v_descale=float("nan")), dict(k_descale=float("inf"))):
        assert status(A, op, **bad) == arg, bad
    for bad in (dict(k=0x1008), dict(v_cache=0x4008), dict(page_table=0x5002), dict(seqlens=0x6001), dict(cu_seqlens=0x7002)):
        assert status(A, op, **bad) == align, bad


def test_rotation_refusals(A):
    p = dict(positions=0x8000, inv_freq=0x9000, rot_dim=64)
    assert status(A, "write", **p) == A.ATTN_OK
    assert status(A, "write", **{**p, "positions": None}) == A.ATTN_ERR_NULL_PTR
    assert status(A, "write", **{**p, "inv_freq": None}) == A.ATTN_ERR_NULL_PTR
    for bad in (dict(rot_dim=-2), dict(rot_dim=63), dict(rot_dim=130), dict(rot_begin=66), dict(rot_begin=-1)):
        assert status(A, "write", **{**p, **bad}) == A.ATTN_ERR_BAD_SHAPE, bad
    for bad in (dict(interleaved=3), dict(amplitude=float("inf"))):
        assert status(A, "write", **{**p, **bad}) == A.ATTN_ERR_BAD_ARG, bad
    for bad in (dict(positions=0x8001), dict(inv_freq=0x9004)):
        assert status(A, "write", **{**p, **bad}) == A.ATTN_ERR_ALIGN, bad


# ------------------------------------------------------------------------------------- GPU

class Cache:
    """A paged cache of random codes, its table (unused entries out of range) and the packed rows."""

    def __init__(self, fmt, Hkv, d, page, n, lens, seed, tail=3, dense=False):
        rs = np.random.RandomState(seed)
        self.fmt, self.Hkv, self.d, self.page, self.B = fmt, Hkv, d, page, len(n)
        self.n, self.lens = np.array(n), np.array(lens)
        pages = -(-self.lens // page)
        self.num, self.width = int(pages.sum()) + 2, int(max(1, pages.max()))
        perm, self.pt, at = rs.permutation(self.num), np.full((self.B, self.width), 2**31 - 1, np.int32), 0
        for b, c in enumerate(pages):
            self.pt[b, :c] = perm[at:at + c]
            at += c
        self.T = int(self.n.sum()) + (0 if dense else tail)
        self.cu = None if dense else torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
        t = torch.bfloat16 if fmt == "bf16" else torch.uint8
        shape = (self.num, page, Hkv, d)
        self.kc, self.vc = (torch.from_numpy(rs.randint(0, 120, shape).astype(np.uint8)).to(DEV).to(t) for _ in range(2))
        # rows strided out of a wider projection
        self.x = torch.from_numpy(rs.standard_normal((self.T, 2 * Hkv * d + 8)) * 3).to(DEV).bfloat16()
        self.k, self.v = self.x[:, :Hkv * d], self.x[:, Hkv * d:2 * Hkv * d]
        self.ptd, self.lend = torch.from_numpy(self.pt).to(DEV), torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        self.kds, self.vds = (1.0, 1.0) if fmt == "bf16" else (0.013, 0.11)

    def rows(self):
        """cache row of every packed row of the sequences"""
        out = []
        for b in range(self.B):
            at = np.arange(self.lens[b] - self.n[b], self.lens[b])
            out.append(self.pt[b, at // self.page].astype(np.int64) * self.page + at % self.page)
        return np.concatenate(out) if out else np.zeros(0, np.int64)

    def write(self, A, **kw):
        A.attn_kv_write_paged(self.k, self.v, self.x.stride(0), self.x.stride(0), self.kc, self.vc, self.ptd, self.lend, self.cu,
                              self.page, self.T, self.B, self.Hkv, self.d, self.width, self.num, self.fmt, self.kds, self.vds, **kw)

    def values(self, cache):
        """decoded codes, without the descale, as float64 [rows, Hkv, d]"""
        if self.fmt == "bf16":
            v = cache
        else:
            v = cache.view(torch.float8_e4m3fn if self.fmt == "e4m3" else torch.float8_e5m2)
        return v.to(torch.float64).cpu().numpy().reshape(-1, self.Hkv, self.d)


def half_step(x, fmt):
    """Half the distance of neighbouring values of the format at |x| (upper neighbourhood)."""
    if fmt == "bf16":
        return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 1e-300))) - 8)
    bits, least, _ = F8[fmt]
    return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), least) - bits - 1)


LAYOUTS = [  # format, Hkv, d, page, rows, lengths, dense
    ("e4m3", 2, 128, 16, [1], [1], True),
    ("e4m3", 8, 128, 16, [1] * 40, list(range(1, 41)), True),
    ("e5m2", 3, 64, 7, [5, 0, 1, 33, 0, 2], [5, 0, 8, 40, 9, 700], False),
    ("bf16", 1, 256, 1, [3, 4], [3, 50], False),
    ("bf16", 5, 16, 100, [17, 17], [17, 99], True),
    ("e4m3", 1, 80, 64, [2000, 1, 900], [2100, 1, 900], False),   # several tokens per block
    ("e5m2", 2, 128, 3, [1] * 70, [3] * 70, False),               # more sequences than one probe of a warp
    ("e4m3", 1, 16, 2, [1] * 1500, [2] * 1500, False),            # two rounds of probes
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,Hkv,d,page,n,lens,dense", LAYOUTS)
@pytest.mark.parametrize("rot,begin,inter", [(0, 0, 0), (16, 0, 0), (16, 0, 1), (6, 3, 0)])
def test_write_then_read(A, fmt, Hkv, d, page, n, lens, dense, rot, begin, inter):
    c = Cache(fmt, Hkv, d, page, n, lens, seed=d + page + rot, dense=dense)
    before = [x.clone() for x in (c.kc, c.vc)]
    pos = np.random.RandomState(1).randint(0, 100000, c.T)
    amp = 1.25
    inv = np.array(A.attn_rope_freqs(rot)[0]) if rot else None
    kw = dict(positions=torch.from_numpy(pos.astype(np.int32)).to(DEV), inv_freq=torch.from_numpy(inv).to(DEV), rot_begin=begin,
              rot_dim=rot, interleaved=inter, amplitude=amp) if rot else {}
    c.write(A, **kw)
    assert A.attn_get_device_status() == 0
    rows, T = c.rows(), int(c.n.sum())
    rest = np.setdiff1d(np.arange(c.num * page), rows)
    for x, cache, old, ds, turned in ((c.k, c.kc, before[0], c.kds, rot > 0), (c.v, c.vc, before[1], c.vds, False)):
        ref = x.double().cpu().numpy()[:T].reshape(T, Hkv, d)
        bound = np.zeros_like(ref)
        if turned:
            ref, bound = rope_reference(ref, pos[:T], inv, begin, rot, inter, 0, amp)
        ds = float(np.float32(ds))
        ref, bound = ref / ds, bound / ds
        bound = bound + 2.0**-23 * np.abs(ref)  # the quotient in fp32
        got = c.values(cache)[rows]
        if fmt != "bf16":
            ref = np.clip(ref, -F8[fmt][2], F8[fmt][2])
        assert (np.abs(got - ref) <= half_step(np.abs(ref) + bound, fmt) + bound).all()
        flat = cache.reshape(c.num * page, -1), old.reshape(c.num * page, -1)
        assert torch.equal(flat[0][rest], flat[1][rest])  # slots of no row are left as they were
    # and back: descale * value, rounded once to bf16 (half a step, 2^-8 relative)
    k, v = (torch.full((c.T, Hkv * d + 16), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    A.attn_kv_read_paged(c.kc, c.vc, k, v, k.stride(0), v.stride(0), c.ptd, c.lend, c.cu, page, c.T, c.B, Hkv, d, c.width, c.num, fmt,
                         c.kds, c.vds)
    assert A.attn_get_device_status() == 0
    for y, cache, ds in ((k, c.kc, c.kds), (v, c.vc, c.vds)):
        ref = c.values(cache)[rows] * float(np.float32(ds))
        got = y[:T, :Hkv * d].double().cpu().numpy().reshape(ref.shape)
        assert (np.abs(got - ref) <= 2.0**-8 * np.abs(ref) * (0 if fmt == "bf16" else 1)).all()
        assert (y[:T, Hkv * d:] == 7).all() and (y[T:] == 7).all()  # gaps and rows behind the last sequence


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_code_round_trips(A, fmt):
    """All finite codes, read as bf16 (exact with a power-of-two descale) and written again, come back."""
    c = Cache(fmt, 1, 128, 2, [2], [2], seed=1, dense=True)
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    for cache in (c.kc, c.vc):
        cache.view(-1)[(c.rows()[0] * 128):(c.rows()[0] + 2) * 128] = codes
    if c.rows()[1] != c.rows()[0] + 1:
        pytest.fail("one page holds both rows")
    k, v = (torch.empty((2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    args = (c.ptd, c.lend, None, 2, 2, 1, 1, 128, c.width, c.num, fmt, 0.5, 2.0)
    A.attn_kv_read_paged(c.kc, c.vc, k, v, 128, 128, *args)
    vals = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float()
    plain = dict(nan=9e9, posinf=8e9, neginf=-8e9)
    assert torch.equal(k.float().view(-1).nan_to_num(**plain), (vals * 0.5).nan_to_num(**plain))
    kc, vc = torch.zeros_like(c.kc), torch.zeros_like(c.vc)
    A.attn_kv_write_paged(k, v, 128, 128, kc, vc, *args)
    fin = torch.isfinite(vals)
    for cache in (kc, vc):
        got = cache.view(-1)[(c.rows()[0] * 128):(c.rows()[0] + 2) * 128]
        assert torch.equal(got[fin], codes[fin])
        back = got.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float()
        assert torch.isnan(back[torch.isnan(vals)]).all()
        assert (back[torch.isinf(vals)].abs() == F8[fmt][2]).all()  # infinities saturate


@pytest.mark.gpu
def test_bad_lengths_pages_and_offsets(A):
    """Each is recorded, writes nothing, and reads zeros (or leaves rows of no sequence alone)."""
    bad = A.ATTN_ERR_DEVICE_BAD_INDEX

    def fresh():
        return Cache("e4m3", 2, 64, 4, [3, 2, 4], [9, 2, 30], seed=5)

    def run(c, zero, keep, written):
        before = c.kc.clone()
        c.write(A)
        assert A.attn_get_device_status() == bad
        rows = c.rows()
        touched = (c.kc != before).view(c.num * c.page, -1).any(1).cpu().numpy()
        assert set(np.flatnonzero(touched)) <= set(rows[written])
        k = torch.full((c.T, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        v = k.clone()
        A.attn_kv_read_paged(c.kc, c.vc, k, v, 128, 128, c.ptd, c.lend, c.cu, c.page, c.T, c.B, 2, 64, c.width, c.num, "e4m3", 1.0, 1.0)
        assert A.attn_get_device_status() == bad
        for y in (k, v):
            assert (y[zero] == 0).all() and (y[keep] == 7).all()
            got = [r for r in range(9) if r not in zero and r not in keep]
            assert (y[got] != 7).any(1).all()

    c = fresh()  # length below the rows
    c.lend[0] = 2
    run(c, [0, 1, 2], [9, 10, 11], [3, 4, 5, 6, 7, 8])
    c = fresh()  # length above the table, negative length
    c.lend[0], c.lend[1] = c.width * c.page + 1, -5
    run(c, [0, 1, 2, 3, 4], [9, 10, 11], [5, 6, 7, 8])
    c = fresh()  # page indices out of range on both sides: tokens 8 (row 2) and 28, 29 (rows 7, 8)
    c.ptd[0, 2], c.ptd[2, 7] = -1, c.num
    run(c, [2, 7, 8], [9, 10, 11], [0, 1, 3, 4, 5, 6])
    c = fresh()  # the last sequence passes the rows: treated as empty
    c.cu[3] = c.T + 1
    run(c, [], list(range(5, c.T)), [0, 1, 2, 3, 4])


@pytest.mark.gpu
def test_rows_before_the_first_sequence(A):
    """Offsets are absolute rows: a call on the later sequences ignores the rows before them."""
    c = Cache("e5m2", 2, 64, 4, [3, 2, 4], [9, 2, 30], seed=6)
    before = c.kc.clone()
    args = (c.ptd[1:], c.lend[1:], c.cu[1:], 4, c.T, 2, 2, 64, c.width, c.num, "e5m2", c.kds, c.vds)
    A.attn_kv_write_paged(c.k, c.v, c.x.stride(0), c.x.stride(0), c.kc, c.vc, *args)
    k = torch.full((c.T, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    A.attn_kv_read_paged(c.kc, c.vc, k, v, 128, 128, *args)
    assert A.attn_get_device_status() == 0
    touched = np.flatnonzero((c.kc != before).view(c.num * 4, -1).any(1).cpu().numpy())
    assert set(touched) <= set(c.rows()[3:])
    assert (k[:3] == 7).all() and (k[9:] == 7).all() and (k[3:9] != 7).any(1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("descale", [1e-38, 2.0**-126, 1e38, -0.02, 3e-39])
def test_extreme_descales(A, descale):
    """The quotient holds where a reciprocal would leave the range of fp32, and for negative factors."""
    c = Cache("e4m3", 1, 64, 4, [4], [4], seed=7, dense=True)
    ds = float(np.float32(descale))
    c.x.copy_((torch.randn(c.x.shape, dtype=torch.float64) * 50 * abs(ds)).bfloat16())
    c.kds = c.vds = descale
    c.write(A)
    ref = c.k.double().cpu().numpy().reshape(4, 1, 64) / ds
    got = c.values(c.kc)[c.rows()]
    ref = np.clip(ref, -448, 448)
    assert (np.abs(got - ref) <= half_step(np.abs(ref) * (1 + 2.0**-23), "e4m3") + 2.0**-23 * np.abs(ref)).all()


@pytest.mark.gpu
def test_write_on_a_side_stream_in_a_graph(A):
    """Captured and replayed: the replay follows new rows and new lengths."""
    c = Cache("e4m3", 4, 128, 16, [1] * 6, [5, 17, 1, 16, 33, 40], seed=9, dense=True)
    inv = torch.tensor(A.attn_rope_freqs(128)[0], dtype=torch.float64, device=DEV)
    kw = dict(positions=c.lend, inv_freq=inv, rot_dim=128)
    c.write(A, **kw)
    want = c.kc.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.write(A, **kw)
    c.kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    rows = torch.from_numpy(c.rows()).to(DEV)
    assert torch.equal(c.kc.view(-1, 512)[rows], want.view(-1, 512)[rows])
    c.x.copy_(torch.randn_like(c.x))
    c.lend.copy_(c.lend - (c.lend > 1).int())
    g.replay()
    torch.cuda.synchronize()
    again = c.kc.clone()
    c.write(A, **kw)
    assert torch.equal(again, c.kc) and A.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
def test_cache_offsets_beyond_32_bits(A, fmt):
    """Rows on the last pages of a cache of more than 2^31 elements, out of rows further apart than that."""
    Hkv, d, page, B, n = 8, 128, 16, 3, 5
    num = 2**31 // (page * Hkv * d) + 9
    t = torch.bfloat16 if fmt == "bf16" else torch.uint8
    kc, vc = (torch.empty((num, page, Hkv, d), dtype=t, device=DEV) for _ in range(2))
    pt = torch.tensor([[num - 1, 0], [num - 2, num - 5], [1, num - 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([9, 20, 32], dtype=torch.int32, device=DEV)
    stride = 2**28 + 8
    x = torch.empty(B * n * stride, dtype=torch.bfloat16, device=DEV)
    k = x.as_strided((B * n, Hkv * d), (stride, 1))
    k.copy_(torch.randn(B * n, Hkv * d))
    v = torch.randn(B * n, Hkv * d, device=DEV).bfloat16()
    A.attn_kv_write_paged(k, v, stride, Hkv * d, kc, vc, pt, lens, None, page, B * n, B, Hkv, d, 2, num, fmt, 0.5, 0.25)
    at = [(int(pt[b, i // page]), i % page) for b in range(B) for i in range(int(lens[b]) - n, int(lens[b]))]
    for cache, y, ds in ((kc, k, 0.5), (vc, v, 0.25)):
        got = torch.stack([cache[p, o] for p, o in at]).view(B * n, -1)
        want = y if fmt == "bf16" else (y.float() / ds).to(torch.float8_e5m2).view(torch.uint8)
        assert torch.equal(got, want)
    k2, v2 = torch.empty_like(v), torch.empty_like(v)
    k.zero_()
    A.attn_kv_read_paged(kc, vc, k, v2, stride, Hkv * d, pt, lens, None, page, B * n, B, Hkv, d, 2, num, fmt, 0.5, 0.25)
    A.attn_kv_read_paged(kc, vc, k2, v2, Hkv * d, Hkv * d, pt, lens, None, page, B * n, B, Hkv, d, 2, num, fmt, 0.5, 0.25)
    assert torch.equal(k, k2) and A.attn_get_device_status() == 0
    want = v if fmt == "bf16" else ((v.float() / 0.25).to(torch.float8_e5m2).float() * 0.25).bfloat16()
    assert torch.equal(v2, want)
