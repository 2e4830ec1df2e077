"""attn_qk_norm_rope and its gradient: refusals on the CPU; on the GPU every element against 64-bit arithmetic with a
bound that counts the roundings, the gradient against the formula's and against differences."""
import numpy as np
import pytest

from helpers import ensure_built
from test_rope import reference as rope_reference

torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def A():
    ensure_built()
    import exact_softmax_attention_gb300 as mod
    return mod


# ------------------------------------------------------------------------------------- CPU

def status(A, back=False, **kw):
    a = dict(q=0x1000, k=0x2000)
    a.update(dict(dq_out=0x3000, dk_out=0x4000) if back else dict(q_out=0x3000, k_out=0x4000))
    a.update(q_weight=0x7000, k_weight=0x7800, eps=1e-6, positions=0x5000, inv_freq=0x6000)
    if back:
        a.update(dq=0x8000, dk=0x9000, dq_weight=None, dk_weight=None)
    a.update(T=0, Hq=4, Hk=2, d=64, rot_begin=0, rot_dim=64, q_stride=256, k_stride=128)
    a.update(dict(dq_out_stride=256, dk_out_stride=128, dq_stride=256, dk_stride=128) if back else dict(q_out_stride=256, k_out_stride=128))
    a.update(elem_type="bf16", interleaved=0, amplitude=1.0)
    a.update(kw)
    f = A.attn_qk_norm_rope_bwd if back else A.attn_qk_norm_rope
    return f(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("back", [False, True])
def test_refusals(A, back):
    null, shape, align, arg = A.ATTN_ERR_NULL_PTR, A.ATTN_ERR_BAD_SHAPE, A.ATTN_ERR_ALIGN, A.ATTN_ERR_BAD_ARG
    assert status(A, back) == A.ATTN_OK  # no rows: nothing to launch
    outs = ("dq", "dk", "dq_out", "dk_out") if back else ("q_out", "k_out")
    for name in ("q", "k", "positions", "inv_freq") + outs:
        assert status(A, back, **{name: None}) == null, name
    none = {x: None for x in outs if "k" in x}
    assert status(A, back, k=None, Hk=0, **none) == A.ATTN_OK
    assert status(A, back, q_weight=None, k_weight=None) == A.ATTN_OK
    assert status(A, back, rot_dim=0, positions=None, inv_freq=None) == A.ATTN_OK
    for bad in (dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(d=63), dict(d=0), dict(d=2048), dict(rot_dim=-2), dict(rot_dim=3),
                dict(rot_dim=66), dict(rot_begin=2), dict(rot_begin=-2, rot_dim=32), dict(q_stride=-1), dict(k_stride=-8), dict(Hq=65536)):
        assert status(A, back, **bad) == shape, bad
    for bad in (dict(elem_type=2), dict(interleaved=2), dict(amplitude=float("nan")), dict(eps=-1e-6), dict(eps=float("inf")),
                dict(eps=float("nan"))):
        assert status(A, back, **bad) == arg, bad
    for bad in (dict(q=0x1001), dict(k=0x2002, elem_type="f32"), dict(positions=0x5002), dict(inv_freq=0x6004), dict(q_weight=0x7002),
                dict(k_weight=0x7801)):
        assert status(A, back, **bad) == align, bad
    if back:
        for bad in (dict(dq_stride=255), dict(dk_stride=127), dict(dq_out_stride=-1), dict(dq=0x3000, dq_stride=512),
                    dict(dk=0x2000, dk_stride=512)):
            assert status(A, back, **bad) == shape, bad
        assert status(A, back, dq_weight=0xa002) == align
        assert status(A, back, k=None, Hk=0, dk_weight=0xa000, **none) == arg
    else:
        for bad in (dict(q_out_stride=255), dict(k_out_stride=127), dict(q_out=0x1000, q_stride=512)):
            assert status(A, back, **bad) == shape, bad


# ------------------------------------------------------------------------------------- GPU

class Problem:
    def __init__(self, A, T, Hq, Hk, d, begin, rot, inter, et, weights, seed=0, far=100000, scale=1.0):
        rs = np.random.RandomState(seed + T + d + rot + inter)
        self.T, self.Hq, self.Hk, self.d, self.begin, self.rot, self.inter, self.et = T, Hq, Hk, d, begin, rot, inter, et
        t = torch.bfloat16 if et == "bf16" else torch.float32
        self.t, self.eps = t, 1e-3
        self.fused = torch.from_numpy(rs.standard_normal((T, (Hq + Hk) * d + 16)) * scale).to(DEV).to(t)  # q and k side by side, and a gap
        self.q, self.k = self.fused[:, :Hq * d], self.fused[:, Hq * d:(Hq + Hk) * d]
        self.pos = rs.randint(-far, far, T)
        self.pos[0] = 0
        freqs, self.amp = A.attn_rope_freqs(rot, 10000.0, "yarn", 4.0, 4096.0) if rot else ([], 1.0)
        self.inv = np.array(freqs)
        self.posd = torch.from_numpy(self.pos.astype(np.int32)).to(DEV)
        self.invd = torch.from_numpy(self.inv).to(DEV)
        self.wq, self.wk = (torch.from_numpy((1 + 0.5 * rs.standard_normal(d)).astype(np.float32)).to(DEV) if weights else None for _ in range(2))
        self.gq, self.gk = (torch.from_numpy(rs.standard_normal((T, h * d + 8))).to(DEV).to(t) for h in (Hq, Hk))

    def forward(self, A, q=None, k=None, qo=None, ko=None, **kw):
        q, k = self.q if q is None else q, self.k if k is None else k
        qo = torch.full((self.T, self.Hq * self.d), float("nan"), dtype=self.t, device=DEV) if qo is None else qo
        ko = torch.full((self.T, self.Hk * self.d + 8), float("nan"), dtype=self.t, device=DEV) if ko is None else ko
        A.attn_qk_norm_rope(q, k, qo, ko, self.wq, self.wk, self.eps, self.posd if self.rot else None, self.invd if self.rot else None, self.T,
                            self.Hq, self.Hk, self.d, self.begin, self.rot, q.stride(0), k.stride(0), qo.stride(0), ko.stride(0), self.et,
                            self.inter, self.amp, **kw)
        return qo, ko

    def backward(self, A, gq=None, gk=None, dq=None, dk=None, sums=True, **kw):
        gq, gk = self.gq if gq is None else gq, self.gk if gk is None else gk
        dq = torch.full((self.T, self.Hq * self.d), float("nan"), dtype=self.t, device=DEV) if dq is None else dq
        dk = torch.full((self.T, self.Hk * self.d + 8), float("nan"), dtype=self.t, device=DEV) if dk is None else dk
        dw = [torch.full((self.d,), float("nan"), device=DEV) if sums and h else None for h in (self.Hq, self.Hk)]
        A.attn_qk_norm_rope_bwd(self.q, self.k, gq, gk, self.wq, self.wk, self.eps, self.posd if self.rot else None,
                                self.invd if self.rot else None, dq, dk, *dw, self.T, self.Hq, self.Hk, self.d, self.begin, self.rot,
                                self.q.stride(0), self.k.stride(0), gq.stride(0), gk.stride(0), dq.stride(0), dk.stride(0), self.et,
                                self.inter, self.amp, **kw)
        return dq, dk, dw

    def turn(self, x, transpose):
        """(rotated, bound of an fp32 evaluation)"""
        if not self.rot:
            return x, np.zeros_like(x)
        return rope_reference(x, self.pos, self.inv, self.begin, self.rot, self.inter, transpose, self.amp)

    def heads(self, i):
        """x [T, H, d], weight, gradient of the output, in 64 bits; the factor of the norm."""
        H = (self.Hq, self.Hk)[i]
        x = (self.q, self.k)[i].double().cpu().numpy().reshape(self.T, H, self.d)
        w = (self.wq, self.wk)[i]
        w = np.ones(self.d) if w is None else w.double().cpu().numpy()
        g = (self.gq, self.gk)[i][:, :H * self.d].double().cpu().numpy().reshape(self.T, H, self.d)
        return x, w, g, 1 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float32(self.eps))


STEP = {"bf16": 2.0**-8, "f32": 2.0**-24}


def norm_error(d):
    """Relative error of an fp32 x w r: the sum of d squares is off by d 2^-24 at most (all terms positive), half of that after
    the root; mean, eps and rsqrt within 4 ulp (2^-22), two products."""
    return (d / 2 + 8) * 2.0**-24


CASES = [  # T, Hq, Hk, d, begin, rot, interleaved, type, weights
    (1, 1, 0, 64, 0, 64, 0, "bf16", True),
    (7, 4, 2, 128, 0, 128, 0, "bf16", True),
    (5, 3, 1, 128, 0, 128, 1, "bf16", False),
    (33, 2, 2, 192, 128, 64, 0, "bf16", True),   # three items per lane
    (33, 2, 3, 192, 128, 64, 1, "f32", True),
    (9, 2, 1, 80, 16, 48, 0, "bf16", True),
    (9, 2, 1, 96, 0, 96, 1, "bf16", True),
    (11, 5, 1, 160, 0, 32, 0, "f32", True),      # idle places
    (9, 2, 1, 80, 3, 10, 0, "bf16", True),       # odd begin: element by element
    (9, 2, 1, 80, 3, 10, 1, "f32", False),
    (4, 1, 1, 2, 0, 2, 0, "f32", True),
    (6, 2, 2, 34, 0, 0, 0, "bf16", True),        # norms only
    (300, 3, 2, 64, 0, 0, 0, "f32", True),
    (3, 2, 1, 1024, 0, 1024, 0, "f32", True),    # four items per lane
    (3, 2, 1, 1024, 512, 512, 1, "bf16", True),
    (5, 1, 1, 1022, 0, 1022, 0, "bf16", True),
    (2600, 2, 1, 64, 0, 32, 0, "bf16", True),    # the last block ragged
    (2501, 1, 1, 256, 0, 24, 1, "f32", True),
    (1201, 7, 3, 128, 0, 128, 0, "bf16", True),  # more heads than groups share evenly
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d,begin,rot,inter,et,weights", CASES)
def test_forward(A, T, Hq, Hk, d, begin, rot, inter, et, weights):
    p = Problem(A, T, Hq, Hk, d, begin, rot, inter, et, weights)
    out = p.forward(A)
    for i, H in ((0, Hq), (1, Hk)):
        if H == 0:
            continue
        x, w, _, r = p.heads(i)
        ref, bound = p.turn(x * r * w, 0)
        size = np.abs(p.turn(np.abs(x * r * w), 0)[1]) / (np.pi * 2.0**-25) + np.abs(ref)  # at least amplitude (|u| + |w|)
        got = out[i][:, :H * d].double().cpu().numpy().reshape(ref.shape)
        bound = bound + size * norm_error(d)
        tol = bound + STEP[et] * (np.abs(ref) + bound) + 1e-38
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    if Hk:
        assert torch.isnan(out[1][:, Hk * d:].float()).all()  # the gap between output rows is left as it was
    qi, ki = p.fused.clone()[:, :Hq * d], p.fused.clone()[:, Hq * d:(Hq + Hk) * d]
    p.forward(A, qi, ki, qi, ki)  # in place
    assert torch.equal(qi, out[0]) and torch.equal(ki, out[1][:, :Hk * d])


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d,begin,rot,inter,et,weights", CASES)
def test_gradient(A, T, Hq, Hk, d, begin, rot, inter, et, weights):
    p = Problem(A, T, Hq, Hk, d, begin, rot, inter, et, weights, seed=1)
    dq, dk, dw = p.backward(A)
    for i, (H, dx) in enumerate(((Hq, dq), (Hk, dk))):
        if H == 0:
            continue
        x, w, dy, r = p.heads(i)
        g, off = p.turn(dy, 1)
        n = x * r
        ref = r * (w * g - n * (n * w * g).mean(-1, keepdims=True))
        # dot product: d roundings of terms that may cancel, n as in the forward pass
        e = norm_error(d)
        dot = (np.abs(n * w * g) * (2 * e + (d + 4) * 2.0**-24) + np.abs(n * w) * off).mean(-1, keepdims=True)
        bound = r * (np.abs(w) * off + np.abs(w * g) * 2 * e + np.abs(n) * (dot + np.abs((n * w * g).mean(-1, keepdims=True)) * 4 * e))
        got = dx[:, :H * d].double().cpu().numpy().reshape(ref.shape)
        tol = bound + STEP[et] * (np.abs(ref) + bound) + 1e-38
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
        # the weights' gradient: no term passes more than T H additions
        ref = (n * g).sum((0, 1))
        tol = (np.abs(n * g) * (e + (T * H + 2) * 2.0**-24) + np.abs(n) * off).sum((0, 1))
        got = dw[i].double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    if Hk:
        assert torch.isnan(dk[:, Hk * d:].float()).all()
    again = p.backward(A)
    assert torch.equal(again[0], dq) and all(torch.equal(a, b) for a, b in zip(again[2], dw) if a is not None)  # the same bytes
    gq, gk = p.gq.clone(), p.gk.clone()  # in place, and without the weights' gradient
    p.backward(A, gq, gk, gq, gk, sums=False)
    assert torch.equal(gq[:, :Hq * d], dq) and torch.equal(gk[:, :Hk * d], dk[:, :Hk * d])
    assert torch.equal(gq[:, Hq * d:], p.gq[:, Hq * d:])


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,et", [(1216, 1024, "f32"), (4864, 512, "bf16"), (1300, 1022, "f32")])
def test_gradient_of_wide_heads_with_many_angles(A, T, d, et):
    """Rows of wide heads for the weights' sums next to the angles of as many tokens as a block takes."""
    test_gradient(A, T, 1, 0, d, 0, d, 0, et, True)


@pytest.mark.gpu
def test_gradient_by_differences(A):
    """<dL/dx, v> and <dL/dw, u> against central differences of the forward call."""
    T, Hq, Hk, d, h = 6, 2, 1, 64, 2.0**-5
    p = Problem(A, T, Hq, Hk, d, 16, 32, 0, "f32", True, seed=2)
    p.fused = p.fused[:, :(Hq + Hk) * d].contiguous()
    p.q, p.k = p.fused[:, :Hq * d], p.fused[:, Hq * d:]
    dq, dk, dw = p.backward(A)
    rs = np.random.RandomState(5)
    v = torch.from_numpy(rs.standard_normal(p.q.shape).astype(np.float32)).to(DEV)
    u = torch.from_numpy(rs.standard_normal(d).astype(np.float32)).to(DEV)

    def loss(q, wq):
        keep, p.wq = p.wq, wq
        y = p.forward(A, q=q.contiguous())[0]
        p.wq = keep
        return (y.double() * p.gq[:, :Hq * d].double()).sum().item()

    def loss64(q, wq):
        x = q.double().cpu().numpy().reshape(T, Hq, d)
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float32(p.eps)) * wq.double().cpu().numpy()
        return (p.turn(y, 0)[0] * p.gq[:, :Hq * d].double().cpu().numpy().reshape(T, Hq, d)).sum()

    x, w, g, r = p.heads(0)
    noise = (np.abs(p.turn(np.abs(x * r * w), 0)[0]).max() * 2 * np.abs(g).sum()) * (norm_error(d) + 2.0**-21) / h  # both evaluations' roundings
    for plus, minus, grad in (((p.q + h * v, p.wq), (p.q - h * v, p.wq), (dq.double() * v.double()).sum().item()),
                              ((p.q, p.wq + h * u), (p.q, p.wq - h * u), (dw[0].double() * u.double()).sum().item())):
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        diff64 = (loss64(*plus) - loss64(*minus)) / (2 * h)
        assert abs(diff - diff64) <= noise
        small = [(loss64(p.q.double() + s * e * v.double(), p.wq.double() + s * (1 - e) * u.double())) for s in (1e-5, -1e-5)
                 for e in ((1,) if plus[1] is p.wq else (0,))]
        assert abs((small[0] - small[1]) / 2e-5 - grad) <= noise * h + 1e-6 * np.abs(g).sum()


@pytest.mark.gpu
def test_zero_heads_extremes_and_empty_calls(A):
    """Heads of zeros give zeros (and finite gradients) for eps > 0; large and small magnitudes; a call without rows."""
    p = Problem(A, 9, 2, 1, 128, 0, 128, 0, "f32", True, seed=3)
    p.fused[2] = 0
    qo, _ = p.forward(A)
    dq, dk, dw = p.backward(A)
    assert (qo[2] == 0).all() and torch.isfinite(dq).all() and torch.isfinite(dw[0]).all()
    for s in (1e-15, 1e15):
        p = Problem(A, 9, 2, 1, 128, 0, 0, 0, "f32", True, seed=3, scale=s)
        p.eps = 0.0
        x, w, _, r = p.heads(0)
        ref = x * r * w
        got = p.forward(A)[0].double().cpu().numpy().reshape(ref.shape)
        assert (np.abs(got - ref) <= np.abs(ref) * (norm_error(128) + 2.0**-24)).all()
    dq, dk, _ = p.backward(A)
    p.T = 0
    assert all((w == 0).all() for w in p.backward(A, dq=dq, dk=dk)[2])  # sums of nothing


@pytest.mark.gpu
def test_streams_graph_and_repeated_rows(A):
    """A side stream, a captured call replayed on new inputs, and inputs of stride 0."""
    p = Problem(A, 700, 4, 2, 128, 0, 128, 0, "bf16", True, seed=4)
    want, grads = p.forward(A), p.backward(A)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gotg = p.forward(A), p.backward(A)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(gotg[0], grads[0]) and torch.equal(gotg[2][1], grads[2][1])
    qo, ko = torch.empty_like(want[0]), torch.empty_like(want[1])
    dq, dk = torch.empty_like(grads[0]), torch.empty_like(grads[1])
    dw = [torch.empty(128, device=DEV) for _ in range(2)]

    def both():
        p.forward(A, qo=qo, ko=ko)
        A.attn_qk_norm_rope_bwd(p.q, p.k, p.gq, p.gk, p.wq, p.wk, p.eps, p.posd, p.invd, dq, dk, *dw, 700, 4, 2, 128, 0, 128, p.q.stride(0),
                                p.k.stride(0), p.gq.stride(0), p.gk.stride(0), dq.stride(0), dk.stride(0), "bf16", 0, p.amp)

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    p.fused.copy_(torch.randn_like(p.fused))
    for x in (qo, dq, *dw):
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    want, grads = p.forward(A), p.backward(A)
    assert torch.equal(qo, want[0]) and torch.equal(dq, grads[0]) and torch.equal(dw[0], grads[2][0]) and torch.equal(dw[1], grads[2][1])
    row = torch.randn((1, 512), device=DEV, dtype=torch.bfloat16)
    many, one = torch.empty((700, 512), device=DEV, dtype=torch.bfloat16), torch.empty((700, 512), device=DEV, dtype=torch.bfloat16)
    for q, stride, out in ((row, 0, many), (row.expand(700, -1).contiguous(), 512, one)):
        A.attn_qk_norm_rope(q, None, out, None, p.wq, None, p.eps, p.posd, p.invd, 700, 4, 0, 128, 0, 128, stride, 0, 512, 0)
    assert torch.equal(many, one)


@pytest.mark.gpu
def test_two_captured_gradients_at_once(A):
    """Graphs with their own parts of the weights' sums, replayed together on two streams."""
    ps = [Problem(A, T, 4, 2, 128, 0, 128, 0, "bf16", True, seed=8) for T in (900, 1700)]
    want = [p.backward(A) for p in ps]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(p.backward(A))
        graphs.append(g)
    for _ in range(5):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (dq, dk, dw), (rq, rk, rw) in zip(got, want):
            assert torch.equal(dq, rq) and torch.equal(dk[:, :256], rk[:, :256]) and torch.equal(dw[0], rw[0]) and torch.equal(dw[1], rw[1])


@pytest.mark.gpu
def test_offsets_beyond_32_bits(A):
    """Rows further apart than 2^31 elements in all, in and out, both ways."""
    T, H, d, stride = 17, 2, 64, 2**27 + 8
    x, y = (torch.empty(T * stride, dtype=torch.bfloat16, device=DEV).as_strided((T, H * d), (stride, 1)) for _ in range(2))
    q, g = (torch.randn(T, H * d, device=DEV).bfloat16() for _ in range(2))
    x.copy_(q)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 1000
    inv = torch.tensor(A.attn_rope_freqs(d)[0], dtype=torch.float64, device=DEV)
    near, w = torch.empty_like(q), torch.rand(d, device=DEV)
    for back in (False, True):
        for src, dst, a, b in ((q, near, H * d, H * d), (x, y, stride, stride)):
            if back:
                A.attn_qk_norm_rope_bwd(src, None, g, None, w, None, 1e-6, pos, inv, dst, None, None, None, T, H, 0, d, 0, d, a, 0, H * d, 0, b, 0)
            else:
                A.attn_qk_norm_rope(src, None, dst, None, w, None, 1e-6, pos, inv, T, H, 0, d, 0, d, a, 0, b, 0)
        assert torch.equal(y, near)


RANGE = [  # d, begin, rot, interleaved, type: two or one items per lane, idle places, element by element
    (128, 0, 128, 0, "bf16"),
    (128, 0, 0, 0, "f32"),
    (192, 128, 64, 1, "f32"),
    (160, 0, 32, 0, "f32"),
    (80, 3, 10, 0, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d,begin,rot,inter,et", RANGE)
@pytest.mark.parametrize("size,grad", [(1e-18, 1e4), (1e-18, 1e-4), (1e17, 1e4), (1e17, 1e-4), (1e-10, 1e19)])
def test_gradient_over_the_range(A, d, begin, rot, inter, et, size, grad):
    """Without eps, heads whose squares, and products with the gradient, fit into fp32 as documented: so does every intermediate value. The
    bound is that of test_gradient, relative to the operands throughout (sums of 10^-36 to 10^34 lose nothing)."""
    T, Hq, Hk = 37, 3, 2
    p = Problem(A, T, Hq, Hk, d, begin, rot, inter, et, True, seed=11, scale=size)
    p.eps = 0.0
    p.gq, p.gk = ((x.double() * grad).to(p.t) for x in (p.gq, p.gk))
    dq, dk, dw = p.backward(A)
    for i, (H, dx) in enumerate(((Hq, dq), (Hk, dk))):
        x, w, dy, r = p.heads(i)
        g, off = p.turn(dy, 1)
        n = x * r
        along = (n * w * g).mean(-1, keepdims=True)
        ref = r * (w * g - n * along)
        e = norm_error(d)
        dot = (np.abs(n * w * g) * (2 * e + (d + 4) * 2.0**-24) + np.abs(n * w) * off).mean(-1, keepdims=True)
        bound = r * (np.abs(w) * off + np.abs(w * g) * 2 * e + np.abs(n) * (dot + np.abs(along) * 4 * e))
        got = dx[:, :H * d].double().cpu().numpy().reshape(ref.shape)
        tol = bound + STEP[et] * (np.abs(ref) + bound) + 1e-38
        assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
        ref = (n * g).sum((0, 1))
        tol = (np.abs(n * g) * (e + (T * H + 2) * 2.0**-24) + np.abs(n) * off).sum((0, 1))
        got = dw[i].double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("d,begin,rot,inter,et", RANGE)
@pytest.mark.parametrize("size,weight", [(1e-18, 1e25), (1e-18, 1e-25), (1e17, 1e30), (1e17, 1e-18)])
def test_forward_over_the_range(A, d, begin, rot, inter, et, size, weight):
    """Weights far from one on small and large heads, without eps; the bound is that of test_forward."""
    T, Hq, Hk = 37, 3, 2
    p = Problem(A, T, Hq, Hk, d, begin, rot, inter, et, True, seed=12, scale=size)
    p.eps = 0.0
    p.wq, p.wk = p.wq * weight, p.wk * weight
    out = p.forward(A)
    for i, H in ((0, Hq), (1, Hk)):
        x, w, _, r = p.heads(i)
        ref, bound = p.turn(x * r * w, 0)
        size_ = np.abs(p.turn(np.abs(x * r * w), 0)[1]) / (np.pi * 2.0**-25) + np.abs(ref)
        got = out[i][:, :H * d].double().cpu().numpy().reshape(ref.shape)
        bound = bound + size_ * norm_error(d)
        tol = bound + STEP[et] * (np.abs(ref) + bound) + 1e-38
        assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("d,begin,rot,inter,et", RANGE)
@pytest.mark.parametrize("T", [5, 900])
def test_gradient_in_the_place_of_the_input(A, d, begin, rot, inter, et, T):
    """dq and dk written over q and k: the same bytes as beside them."""
    p = Problem(A, T, 5, 2, d, begin, rot, inter, et, True, seed=13)
    dq, dk, dw = p.backward(A)
    _, _, again = p.backward(A, dq=p.q, dk=p.k)
    assert torch.equal(p.q, dq) and torch.equal(p.k, dk[:, :2 * d])
    assert all(torch.equal(a, b) for a, b in zip(again, dw))
