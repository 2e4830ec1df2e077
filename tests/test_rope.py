"""attn_rope and attn_rope_freqs: refusals and tables on the CPU; on the GPU the rotation and its
gradient against extended precision, element by element, with a bound that counts the roundings."""
import ctypes
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

def rope_status(A, **kw):
    a = dict(q=0x1000, k=0x2000, q_out=0x3000, k_out=0x4000, positions=0x5000, inv_freq=0x6000, T=0, Hq=4, Hk=2, d=64, rot_begin=0,
             rot_dim=64, q_stride=256, k_stride=128, q_out_stride=256, k_out_stride=128, elem_type="bf16", interleaved=0,
             transpose=0, amplitude=1.0)
    a.update(kw)
    return A.attn_rope(*a.values(), stream=0, raise_on_error=False)


def test_rope_refusals(A):
    ok, null, shape, align, arg = A.ATTN_OK, A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    assert rope_status(A) == ok  # no rows: nothing to launch
    for name in ("q", "q_out", "k", "k_out", "positions", "inv_freq"):
        assert rope_status(A, **{name: None}) == null
    assert rope_status(A, k=None, k_out=None, Hk=0) == ok
    for bad in (dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(d=63), dict(d=0), dict(d=2048, rot_dim=64), dict(rot_dim=0), dict(rot_dim=3),
                dict(rot_dim=66), dict(rot_begin=2), dict(rot_begin=-2, rot_dim=32), dict(q_stride=-1), dict(k_stride=-8),
                dict(q_out_stride=255), dict(k_out_stride=127), dict(q_out=0x1000, q_stride=512), dict(Hq=65536, q_out_stride=1 << 23),
                dict(rot_begin=2**31 - 2)):
        assert rope_status(A, **bad) == shape, bad
    for bad in (dict(elem_type=2), dict(interleaved=2), dict(transpose=-1), dict(amplitude=float("nan")),
                dict(amplitude=float("inf"))):
        assert rope_status(A, **bad) == arg, bad
    for bad in (dict(q=0x1001), dict(q_out=0x3002, elem_type="f32"), dict(k=0x2001), dict(positions=0x5002), dict(inv_freq=0x6004)):
        assert rope_status(A, **bad) == align, bad


def test_rope_freqs_tables(A):
    rot, theta, s, n0 = 64, 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2)
    f = theta ** (-2.0 * i / rot)
    tol = dict(rtol=1e-13, atol=0)  # a few roundings of pow and one division in 64 bits
    got, amp = A.attn_rope_freqs(rot, theta)
    np.testing.assert_allclose(got, f, **tol)
    assert amp == 1.0
    got, amp = A.attn_rope_freqs(rot, theta, "linear", s)
    np.testing.assert_allclose(got, f / s, **tol)
    assert amp == 1.0
    got, _ = A.attn_rope_freqs(rot, theta, "ntk", s)
    np.testing.assert_allclose(got, (theta * s ** (rot / (rot - 2))) ** (-2.0 * i / rot), **tol)
    np.testing.assert_allclose(got[-1], f[-1] / s, **tol)  # the slowest frequency is interpolated in full
    got, amp = A.attn_rope_freqs(rot, theta, "yarn", s, n0, 32.0, 1.0)
    g = np.clip((n0 * f / (2 * math.pi) - 1) / 31, 0, 1)
    np.testing.assert_allclose(got, g * f + (1 - g) * f / s, rtol=1e-12, atol=0)
    assert abs(amp - (0.1 * math.log(s) + 1)) < 1e-15
    assert got[0] == f[0] and abs(got[-1] / (f[-1] / s) - 1) < 1e-13  # the ends are kept and interpolated


def test_rope_freqs_refusals(A):
    out, amp = (ctypes.c_double * 64)(), ctypes.c_double()

    def call(o=out, a=ctypes.byref(amp), rot=64, theta=1e4, scaling=0, factor=1.0, n=0.0, fast=32.0, slow=1.0):
        return A.lib.attn_rope_freqs(o, a, rot, theta, scaling, factor, n, fast, slow)

    assert call() == A.ATTN_OK
    assert call(o=None) == A.ATTN_ERR_NULL_PTR and call(a=None) == A.ATTN_ERR_NULL_PTR
    for rot in (0, -2, 3, 2048):
        assert call(rot=rot) == A.ATTN_ERR_BAD_SHAPE
    assert call(rot=2, scaling=2, factor=2.0) == A.ATTN_ERR_BAD_SHAPE
    for bad in (dict(theta=0.0), dict(theta=float("nan")), dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5),
                dict(scaling=2, factor=float("inf")), dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, n=4096.0, fast=1.0)):
        assert call(**bad) == A.ATTN_ERR_BAD_ARG, bad


# ------------------------------------------------------------------------------------- GPU

def reference(x, positions, inv_freq, begin, rot, interleaved, transpose, amplitude):
    """(y, bound): rotation of x [T, H, d] (float64) in extended precision, and how far an fp32
    evaluation of the same formula may be from it before it is rounded to the output type."""
    turn = 8 * np.arctan(np.longdouble(1))
    angle = np.mod(positions.astype(np.longdouble)[:, None] * inv_freq.astype(np.longdouble), turn)
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    if transpose:
        s = -s
    y, bound = x.copy(), np.zeros_like(x)
    i = np.arange(rot // 2)
    a, b = (begin + 2 * i, begin + 2 * i + 1) if interleaved else (begin + i, begin + i + rot // 2)
    u, w = x[..., a], x[..., b]
    y[..., a], y[..., b] = amplitude * (u * c - w * s), amplitude * (u * s + w * c)
    # angle: f / (2 pi) and its product with 2^64 each round 2^-53 of f, times the position; the
    # phase rounds to fp32 (half turns up to 1: pi 2^-25); sincospi is within 2 ulp (2^-23 below 1);
    # amplitude, two products and the sum round 2^-24 each of terms up to |u| or |w|
    far = np.abs(positions).astype(np.float64)[:, None] * np.abs(inv_freq) * 2.0**-52
    e = far[:, None] + math.pi * 2.0**-25 + 2.0**-23 + 4 * 2.0**-24
    bound[..., a] = bound[..., b] = amplitude * (np.abs(u) + np.abs(w)) * e
    return y, bound


CASES = [  # T, Hq, Hk, d, begin, rot, interleaved, type
    (1, 1, 0, 64, 0, 64, 0, "bf16"),
    (7, 4, 2, 128, 0, 128, 0, "bf16"),
    (5, 3, 1, 128, 0, 128, 1, "bf16"),
    (33, 2, 2, 192, 128, 64, 0, "bf16"),    # the last third of 192-wide heads
    (33, 2, 2, 192, 128, 64, 1, "f32"),
    (9, 2, 1, 80, 16, 48, 0, "bf16"),
    (9, 2, 1, 80, 3, 10, 0, "bf16"),        # odd begin: element by element
    (9, 2, 1, 80, 3, 10, 1, "f32"),
    (4, 1, 1, 2, 0, 2, 0, "f32"),
    (3, 2, 1, 1024, 0, 1024, 0, "f32"),
    (3, 2, 1, 1024, 512, 512, 1, "bf16"),
    (2600, 2, 1, 64, 0, 32, 0, "bf16"),     # several tokens per block, the last block ragged
    (2501, 1, 1, 64, 0, 24, 1, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d,begin,rot,inter,et", CASES)
@pytest.mark.parametrize("transpose", [0, 1])
def test_rope_parity(A, T, Hq, Hk, d, begin, rot, inter, et, transpose):
    rs = np.random.RandomState(T + d + rot + inter)
    t = torch.bfloat16 if et == "bf16" else torch.float32
    eps = 2.0**-8 if et == "bf16" else 2.0**-24
    fused = torch.from_numpy(rs.standard_normal((T, (Hq + Hk) * d + 16))).to(DEV).to(t)  # q and k side by side, and a gap
    q, k = fused[:, :Hq * d], fused[:, Hq * d:(Hq + Hk) * d]
    qo = torch.full((T, Hq * d), float("nan"), dtype=t, device=DEV)
    ko = torch.full((T, Hk * d + 8), float("nan"), dtype=t, device=DEV)
    pos = rs.randint(-(2**31), 2**31, T)
    pos[: T // 2] = rs.randint(0, 40000, T // 2)
    pos[0] = 0
    freqs, amp = A.attn_rope_freqs(rot, 10000.0, "yarn", 4.0, 4096.0)
    inv = np.array(freqs)
    A.attn_rope(q, k, qo, ko, torch.from_numpy(pos.astype(np.int32)).to(DEV), torch.from_numpy(inv).to(DEV), T, Hq, Hk, d, begin, rot,
                fused.stride(0), fused.stride(0), Hq * d, Hk * d + 8, et, inter, transpose, amp)
    for x, y, H in ((q, qo, Hq), (k, ko, Hk)):
        if H == 0:
            continue
        ref, bound = reference(x.double().cpu().numpy().reshape(T, H, d), pos, inv, begin, rot, inter, transpose, amp)
        got = y[:, :H * d].double().cpu().numpy().reshape(T, H, d)
        tol = bound + eps * (np.abs(ref) + bound) + 1e-38
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    assert torch.isnan(ko[:, Hk * d:].float()).all()  # the gap between output rows is left as it was


@pytest.mark.gpu
def test_rope_angles_of_any_frequency(A):
    """cos and sin of position * frequency against exact integers: frequencies above and below one turn, negative,
    tiny and zero, positions over the whole range; non-finite frequencies give NaN in their columns only."""
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10**64)
    freqs = [1.0, 0.5, 2.0**-9, 2.0**-9 - 2.0**-62, 2.0**-10, 3e-5, 1e-12, 1e-18, 1e-300, 5e-324, 0.0, -0.37, 6.283185307179586, 3.0, 1000.123,
             2.0**20 + 0.25, 2.0**60, float("inf"), float("-inf"), float("nan")]
    pos = [0, 1, -1, 7, 4095, 131071, 2**24 + 1, 10**9 + 7, 2**31 - 1, -(2**31)]
    n, T = len(freqs), len(pos)
    x = torch.cat([torch.ones(T, n), torch.zeros(T, n)], 1).to(DEV)
    y = torch.empty_like(x)
    A.attn_rope(x, None, y, None, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(freqs, dtype=torch.float64, device=DEV), T, 1, 0,
                2 * n, 0, 2 * n, 2 * n, 0, 2 * n, 0, "f32")
    y = y.double().cpu().numpy()
    for i, f in enumerate(freqs):
        for t, m in enumerate(pos):
            c, s = y[t, i], y[t, n + i]
            if not math.isfinite(f):
                assert math.isnan(c) and math.isnan(s)
                continue
            # sincospif within 1.5 ulp, the added rotation and the products rounded once each: 4 * 2^-24; the fraction
            # of a turn is cut to 2^-64 and 1 / (2 pi) rounded to 67 bits: (1 + f / 8) 2^-64 turns per position
            tol = 2.0**-22 + 2 * math.pi * abs(m) * (1 + abs(f) / 8) * 2.0**-64
            if tol > 1:
                assert abs(c) <= 1.001 and abs(s) <= 1.001
                continue
            turns = Fraction(f) * m / two_pi
            angle = float((turns - round(turns)) * two_pi)
            assert abs(c - math.cos(angle)) <= tol and abs(s - math.sin(angle)) <= tol, (f, m)


@pytest.mark.gpu
def test_rope_in_place_and_gradient(A):
    """In place gives the same bytes; transpose undoes the rotation and is its gradient by differences."""
    T, H, d, rot = 40, 3, 96, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H * d), generator=g).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 37
    inv = torch.tensor(A.attn_rope_freqs(rot)[0], dtype=torch.float64, device=DEV)

    def rope(x, transpose=0, out=None):
        y = torch.empty_like(x) if out is None else out
        A.attn_rope(x, None, y, None, pos, inv, T, H, 0, d, 32, rot, H * d, 0, H * d, 0, "f32", 0, transpose)
        return y

    y = rope(x)
    z = x.clone()
    assert torch.equal(rope(z, out=z), y)
    # R R^T = 1 within the rounding of cos^2 + sin^2 and the products: 2 (|u| + |w|) (2^-22 + ...) < 2e-6 |x|max
    assert (rope(y, 1) - x).abs().max().item() <= 4e-6 * x.abs().max().item()
    # directional difference: the map is linear, so <g, R(x + h) - R(x)> = <R^T g, h> up to rounding
    gr, h = torch.randn((2, T, H * d), generator=g).to(DEV)
    lhs = (gr.double() * (rope(x + h).double() - y.double())).sum().item()
    rhs = (rope(gr, 1).double() * ((x + h).double() - x.double())).sum().item()
    # each of the T H d terms is off by at most 2^-21 (|x| + |h|) |g|, about N(0,1) values
    assert abs(lhs - rhs) <= T * H * d * 2.0**-21 * 8


@pytest.mark.gpu
def test_rope_stream_and_repeated_rows(A):
    """A side stream and an input of stride 0 (every row the same vector)."""
    T, H, d = 300, 2, 64
    s = torch.cuda.Stream()
    x = torch.randn((1, H * d), device=DEV, dtype=torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv = torch.tensor(A.attn_rope_freqs(d)[0], dtype=torch.float64, device=DEV)
    y, z = (torch.empty((T, H * d), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    torch.cuda.synchronize()
    A.attn_rope(x, None, y, None, pos, inv, T, H, 0, d, 0, d, 0, 0, H * d, 0, stream=s)
    s.synchronize()
    A.attn_rope(x.expand(T, -1).contiguous(), None, z, None, pos, inv, T, H, 0, d, 0, d, H * d, 0, H * d, 0)
    assert torch.equal(y, z) and torch.equal(y[:1], x)


@pytest.mark.gpu
@pytest.mark.parametrize("et", ["bf16", "f32"])
def test_rope_offsets_beyond_32_bits(A, et):
    """Rows further apart than 2^31 elements in all, in and out."""
    T, H, d, stride = 17, 2, 64, 2**27 + 8
    t = torch.bfloat16 if et == "bf16" else torch.float32
    x = torch.empty(T * stride, dtype=t, device=DEV).as_strided((T, H * d), (stride, 1))
    y = torch.empty(T * stride, dtype=t, device=DEV).as_strided((T, H * d), (stride, 1))
    q = torch.randn(T, H * d, device=DEV).to(t)
    x.copy_(q)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 1000
    inv = torch.tensor(A.attn_rope_freqs(d)[0], dtype=torch.float64, device=DEV)
    near = torch.empty_like(q)
    A.attn_rope(q, None, near, None, pos, inv, T, H, 0, d, 0, d, H * d, 0, H * d, 0, et)
    A.attn_rope(x, None, y, None, pos, inv, T, H, 0, d, 0, d, stride, 0, stride, 0, et)
    assert torch.equal(y, near)
