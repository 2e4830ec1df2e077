"""Measured operators: rotary positions, paged key/value cache writes and reads, and attention of a
tree of drafted tokens over a paged cache. ``own`` selects the library's calls or the plain form."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ------------------------------------------------------------------------------------ cases

def _rope(name, tokens, hq, hk, d, rot_begin, rot, interleaved=False, grad=False, f32=False, fused=True, far=32768,
          factor=1.0):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot_begin": rot_begin, "rot": rot,
            "interleaved": interleaved, "grad": grad, "f32": f32, "fused": fused, "far": far, "factor": factor}


def _kv(name, op, B, lo, hi, ctx, hkv, d, page, fmt, rot=0, interleaved=False, lens=1):
    """new (write) or read tokens of each of B sequences: U[lo, hi]; up to ctx tokens before them."""
    return {"name": name, "op": op, "B": B, "lo": lo, "hi": hi, "ctx": ctx, "hkv": hkv, "d": d, "page": page, "fmt": fmt,
            "rot": rot, "interleaved": interleaved, "lens": lens}


def _tree(name, B, n_lo, n_hi, lo, hi, hq, hkv, d, page, fmt, chain=False, lens=1):
    """n new tokens per sequence, U[n_lo, n_hi] (dense rows when equal), after U[lo, hi] cached ones."""
    return {"name": name, "op": "tree", "B": B, "n_lo": n_lo, "n_hi": n_hi, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "fmt": fmt, "chain": chain, "lens": lens}


def listed():
    return [
        # one decode step of a batch of 64: q and k of one token each, read out of the fused projection
        _rope("rope_step", 64, 32, 8, 128, 0, 128),
        # packed prefill of eight prompts, positions interpolated beyond the trained length
        _rope("rope_prefill", 18432, 32, 8, 128, 0, 128, far=131072, factor=4.0),
        # training: gradient through the rotated last third of 192-wide heads, fp32 gradients
        _rope("rope_grad_part", 8192, 16, 16, 192, 128, 64, interleaved=True, grad=True, f32=True, fused=False),
        # one decode step of a batch of 64 into an 8-bit cache, keys rotated on the way
        _kv("write_step", "write", 64, 1, 1, 256, 8, 128, 16, "e4m3", rot=128),
        # packed prompts into an 8-bit cache, keys rotated on the way
        _kv("write_prefill", "write", 8, 512, 4096, 1000, 8, 128, 16, "e4m3", rot=128),
        # drafted tokens of ragged counts, odd pages, narrow heads, no rotation
        _kv("write_ragged", "write", 48, 1, 63, 500, 3, 64, 7, "e5m2"),
        # a cached prefix back to bf16 rows for the forward
        _kv("read_prefix", "read", 64, 256, 8192, 0, 8, 128, 16, "e4m3"),
        # the newest tokens of a few sequences out of a bf16 cache with odd pages
        _kv("read_tail", "read", 5, 1, 40, 900, 3, 64, 7, "bf16"),
        # one user, eight drafted tokens, short context: latency
        _tree("tree_one", 1, 8, 8, 1000, 1000, 32, 8, 128, 16, "bf16"),
        # a serving batch: 16 drafted tokens each over long ragged contexts
        _tree("tree_batch", 64, 16, 16, 1024, 32768, 32, 8, 128, 16, "bf16"),
        # the same over an 8-bit cache
        _tree("tree_batch_e4m3", 64, 16, 16, 1024, 32768, 32, 8, 128, 16, "e4m3"),
        # chains of ragged length, narrow heads, odd pages
        _tree("chain_ragged", 48, 1, 6, 1, 8000, 12, 3, 64, 7, "e5m2", chain=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree"])
    seed = rng.randrange(1 << 20)
    if op == "rope":
        d = rng.choice([64, 128, 192, 256])
        half = rng.choice([d // 2, d // 4, 32, 24])
        rot = 2 * half
        begin = rng.choice([0, d - rot])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 3, 4, 8])
        f32 = rng.random() < 0.3
        most = min(24000, 18432 * 40 * 128 // ((hq + hk) * d * (2 if f32 else 1)))
        c = _rope(None, _log(rng, 1, most), hq, hk, d, begin, rot, rng.random() < 0.4, rng.random() < 0.3, f32,
                  rng.random() < 0.6, rng.choice([4096, 32768, 1000000]), rng.choice([1.0, 4.0, 8.0]))
    elif op in ("write", "read"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 5, 8])
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(8192, 260000 // B))
        lo = rng.choice([1, hi])
        rot = rng.choice([0, d, d // 2]) if op == "write" else 0
        c = _kv(None, op, B, lo, hi, rng.choice([0, 1, 300, 1000]) if op == "write" else 0, hkv, d, rng.choice([1, 7, 16, 16, 64, 256]),
                rng.choice(["bf16", "e4m3", "e5m2"]), rot, rng.random() < 0.4, seed)
    else:
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 3, 4, 8])
        B = _log(rng, 1, 64)
        n_hi = _log(rng, 1, 96)
        n_lo = rng.choice([1, n_hi])
        # no more scores than the largest listed case, nor more cached tokens
        hi = _log(rng, 1, max(1, min(32768, 64 * 32768 * 32 * 16 // (B * hkv * g * n_hi), 64 * 32768 // B)))
        lo = rng.choice([1, hi, max(1, hi // 32)])
        c = _tree(None, B, n_lo, n_hi, lo, hi, hkv * g, hkv, d, rng.choice([1, 7, 16, 16, 64, 256]),
                  rng.choice(["bf16", "bf16", "e4m3", "e5m2"]), rng.random() < 0.3, seed)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ shapes

def _counts(case):
    """(new or read tokens, cached tokens with them) of each sequence; the same for every seed."""
    rs = np.random.RandomState(case["lens"])
    B = case["B"]
    if case["op"] == "tree":
        n = rs.randint(case["n_lo"], case["n_hi"] + 1, B)
        return n, n + rs.randint(case["lo"], case["hi"] + 1, B)
    n = rs.randint(case["lo"], case["hi"] + 1, B)
    return n, n + rs.randint(0, case["ctx"] + 1, B)


def work(case):
    if case["op"] == "rope":
        e = 4 if case["f32"] else 2
        n = case["tokens"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * n * case["d"] * e + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    n, lens = _counts(case)
    e = 2 if case["fmt"] == "bf16" else 1
    pages = -(-lens // case["page"])
    table = 4 * int(pages.sum()) + 8 * len(n)
    if case["op"] == "tree":
        row = case["hkv"] * case["d"]
        bits = 0 if case["chain"] else 8 * int(n.sum()) * (-(-int(n.max()) // 64))
        return {"bytes": 2 * int(lens.sum()) * row * e + int(n.sum()) * case["hq"] * (4 * case["d"] + 4) + table + bits,
                "flops": 4 * int((n * lens).sum()) * case["hq"] * case["d"]}
    one = 2 * int(n.sum()) * case["hkv"] * case["d"]
    return {"bytes": one * (2 + e) + table, "flops": one + 3 * int(n.sum()) * case["hkv"] * case["rot"]}


# ------------------------------------------------------------------------------------ inputs

def _inv_freq(rot, factor, dev):
    """Position interpolation: base 10000, positions divided by `factor`; 64 bits."""
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot) / factor


def _pages(case, lens, rs):
    """Page table of a pool that a seeded permutation hands out, with some pages that no sequence holds."""
    pages = -(-lens // case["page"])
    spare = 3
    num = int(pages.sum()) + spare
    perm = rs.permutation(num).astype(np.int32)
    width = int(pages.max())
    ends = np.cumsum(pages)
    pt = np.full((len(lens), width), -1, dtype=np.int32)
    for b in range(len(lens)):
        pt[b, :pages[b]] = perm[ends[b] - pages[b]:ends[b]]
    return pt, num, width


def _cache(case, num, g):
    """(key cache, value cache, key descale, value descale): values N(0, 1), codes of x / descale."""
    shape = (num, case["page"], case["hkv"], case["d"])
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        if case["fmt"] == "bf16":
            out.append(x)
        else:
            t, big = FP8[case["fmt"]]
            out.append((x.float() * (big / 6.0)).clamp(-big, big).to(t).view(torch.uint8))
    scale = 1.0 if case["fmt"] == "bf16" else float(np.float32(6.0 / FP8[case["fmt"]][1]))
    return out[0], out[1], scale, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}
    if case["op"] == "rope":
        T, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        t = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:  # q, k and v side by side, as the projection leaves them
            x = torch.randn((T, (hq + 2 * hk) * d), generator=g, device=DEV, dtype=t)
            s["q"], s["k"] = x[:, :hq * d], x[:, hq * d:(hq + hk) * d]
        else:
            s["q"] = torch.randn((T, hq * d), generator=g, device=DEV, dtype=t)
            s["k"] = torch.randn((T, hk * d), generator=g, device=DEV, dtype=t)
        s["q_out"] = torch.empty((T, hq, d), dtype=t, device=DEV)
        s["k_out"] = torch.empty((T, hk, d), dtype=t, device=DEV)
        s["positions"] = torch.from_numpy(rs.randint(0, case["far"], T).astype(np.int32)).to(DEV)
        s["inv_freq"] = _inv_freq(case["rot"], case["factor"], DEV)
        return s
    n, lens = _counts(case)
    B, T = len(n), int(n.sum())
    pt, num, width = _pages(case, lens, rs)
    s.update(T=T, B=B, width=width, num=num, max_q=int(n.max()), longest=int(lens.max()))
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).to(DEV)
    s["dense"] = bool((n == n[0]).all())  # equal counts: no offsets needed
    s["page_table"] = torch.from_numpy(pt).to(DEV)
    s["seqlens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
    s["kc"], s["vc"], s["kds"], s["vds"] = _cache(case, num, g)
    if case["op"] == "tree":
        s["q"] = torch.randn((T, case["hq"], case["d"]), generator=g, device=DEV, dtype=torch.bfloat16) * 2
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, case["hq"]), dtype=torch.float32, device=DEV)
        words = -(-s["max_q"] // 64)
        bits = np.zeros((T, words), dtype=np.uint64)
        for b in range(B):
            for i in range(int(n[b])):  # a node's parent is one of the nodes before it, or the context
                p = rs.randint(-1, i) if i else -1
                if p >= 0:
                    bits[cu[b] + i] = bits[cu[b] + p]
                bits[cu[b] + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        s["mask"], s["words"] = (None, 0) if case["chain"] else (torch.from_numpy(bits.view(np.int64)).to(DEV), words)
        return s
    shape = (T, case["hkv"] * case["d"])
    if case["op"] == "write":
        x = torch.randn((T, 2 * shape[1]), generator=g, device=DEV, dtype=torch.bfloat16)
        s["k"], s["v"] = x[:, :shape[1]], x[:, shape[1]:]
        s["positions"] = torch.from_numpy(np.concatenate([np.arange(l - m, l) for m, l in zip(n, lens)]).astype(np.int32)).to(DEV)
        s["inv_freq"] = _inv_freq(case["rot"], 1.0, DEV) if case["rot"] else None
    else:
        s["k"] = torch.empty((T, case["hkv"], case["d"]), dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.empty_like(s["k"])
    return s


# ------------------------------------------------------------------------------------ plain form

def _rotate(x, positions, inv_freq, begin, rot, interleaved, grad):
    """x [T, H, d] in 32 bits; the angles, which reach far positions, in 64."""
    angle = positions.double()[:, None] * inv_freq
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if grad:
        sn = -sn
    part = x[..., begin:begin + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((x[..., :begin], turned, x[..., begin + rot:]), -1)


def _places(s):
    """Sequence, index within the new tokens, and cache row of every packed row."""
    page = s["case"]["page"]
    cu, t = s["cu"].long(), torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    at = s["seqlens"].long()[b] - (cu[b + 1] - cu[b]) + i
    return b, i, s["page_table"][b, at // page].long() * page + at % page


def _decoded(x, fmt, descale):
    return x.float() if fmt == "bf16" else x.view(FP8[fmt][0]).float() * descale


def _as_values(x, fmt):
    return x if fmt == "bf16" else x.view(FP8[fmt][0])


def _write(s):
    c = s["case"]
    k, v = (x.reshape(s["T"], c["hkv"], c["d"]).float() for x in (s["k"], s["v"]))
    if c["rot"]:
        k = _rotate(k, s["positions"], s["inv_freq"], 0, c["rot"], c["interleaved"], False)
    rows = _places(s)[2]
    for x, cache, descale in ((k, s["kc"], s["kds"]), (v, s["vc"], s["vds"])):
        flat = cache.view(-1, c["hkv"], c["d"])
        if c["fmt"] == "bf16":
            flat[rows] = x.bfloat16()
        else:
            t, big = FP8[c["fmt"]]
            flat[rows] = (x / descale).clamp(-big, big).to(t).view(torch.uint8)
    return {"k_cache": _as_values(s["kc"], c["fmt"]), "v_cache": _as_values(s["vc"], c["fmt"])}


def _read(s):
    c = s["case"]
    rows = _places(s)[2]
    k, v = (_decoded(x.view(-1, c["hkv"], c["d"])[rows], c["fmt"], ds).bfloat16()
            for x, ds in ((s["kc"], s["kds"]), (s["vc"], s["vds"])))
    return {"k": k, "v": v}


def _visible(s, b, i, L):
    """[len(b), L]: which cached tokens row i of sequence b sees."""
    cu, lens = s["cu"].long(), s["seqlens"].long()
    key = torch.arange(L, device=DEV)
    n = cu[b + 1] - cu[b]
    j = key - (lens[b] - n)[..., None]  # index among the drafted tokens, negative before them
    if s["mask"] is None:
        return j <= i[..., None]
    row = s["mask"][(cu[b] + i).clamp(max=s["T"] - 1)]
    jc = j.clamp(0, 64 * s["words"] - 1)
    bit = (row.gather(-1, jc // 64) >> (jc % 64)) & 1
    return (j < 0) | ((j < n[..., None]) & (bit == 1))


def _attend(s):
    c = s["case"]
    B, hkv, d, n, L = s["B"], c["hkv"], c["d"], s["max_q"], s["width"] * c["page"]
    G = c["hq"] // hkv
    b, i, _ = _places(s)
    held = (torch.arange(L, device=DEV) < s["seqlens"].long()[:, None])[..., None, None]
    K, V = (torch.where(held, _decoded(x[s["page_table"].clamp(min=0)].view(B, L, hkv, d), c["fmt"], ds), 0.0).transpose(1, 2)
            for x, ds in ((s["kc"], s["kds"]), (s["vc"], s["vds"])))
    q = torch.zeros((B, n, hkv, G, d), device=DEV)
    q[b, i] = s["q"].float().view(-1, hkv, G, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, d)
    score = (q @ K.transpose(2, 3)).view(B, hkv, n, G, L).mul_(1.0 / math.sqrt(d))
    seen = torch.zeros((B, n, L), dtype=torch.bool, device=DEV)
    seen[b, i] = _visible(s, b, i, L)
    score.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, n * G, L) @ V).view(B, hkv, n, G, d) / total.clamp(min=1e-38)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4)[b, i].reshape(-1, c["hq"], d)
    return {"o": o.bfloat16(), "lse": lse.permute(0, 2, 1, 3)[b, i].reshape(-1, c["hq"])}


# ------------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "rope":
        q, k = (_rotate(x.reshape(c["tokens"], h, c["d"]).float(), s["positions"], s["inv_freq"], c["rot_begin"], c["rot"],
                        c["interleaved"], c["grad"]).to(x.dtype) for x, h in ((s["q"], c["hq"]), (s["k"], c["hk"])))
        return {"q": q, "k": k}
    return {"write": _write, "read": _read, "tree": _attend}[c["op"]](s)


def _run_own(s):
    import exact_softmax_attention_gb300 as A

    c = s["case"]
    if c["op"] == "rope":
        A.attn_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["inv_freq"], c["tokens"], c["hq"], c["hk"], c["d"],
                    c["rot_begin"], c["rot"], s["q"].stride(0), s["k"].stride(0), c["hq"] * c["d"], c["hk"] * c["d"],
                    "f32" if c["f32"] else "bf16", c["interleaved"], c["grad"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cu = None if s["dense"] else s["cu"]
    if c["op"] == "tree":
        A.attn_decode_paged_tree(s["q"], s["kc"], s["vc"], s["page_table"], s["seqlens"], cu, s["mask"], s["words"], c["page"],
                                 s["o"], s["lse"], None, s["T"], s["B"], s["max_q"], c["hq"], c["hkv"], c["d"], s["width"],
                                 s["num"], 1.0 / math.sqrt(c["d"]), 0, c["fmt"], s["kds"], s["vds"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "write":
        A.attn_kv_write_paged(s["k"], s["v"], s["k"].stride(0), s["v"].stride(0), s["kc"], s["vc"], s["page_table"],
                              s["seqlens"], cu, c["page"], s["T"], s["B"], c["hkv"], c["d"], s["width"], s["num"], c["fmt"],
                              s["kds"], s["vds"], s["positions"] if c["rot"] else None, s["inv_freq"], 0, c["rot"],
                              c["interleaved"])
        return {"k_cache": _as_values(s["kc"], c["fmt"]), "v_cache": _as_values(s["vc"], c["fmt"])}
    row = c["hkv"] * c["d"]
    A.attn_kv_read_paged(s["kc"], s["vc"], s["k"], s["v"], row, row, s["page_table"], s["seqlens"], cu, c["page"], s["T"],
                         s["B"], c["hkv"], c["d"], s["width"], s["num"], c["fmt"], s["kds"], s["vds"])
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------------------------ 64 bits

def _turned64(x, positions, inv_freq, begin, rot, interleaved, grad):
    """The rotation pair by pair as complex numbers, 64 bits: x [T, H, d]."""
    angle = positions.double().unsqueeze(1).mul(inv_freq) * (-1.0 if grad else 1.0)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    out = x.double().clone()
    first = torch.arange(rot // 2, device=x.device)
    first, second = (begin + 2 * first, begin + 2 * first + 1) if interleaved else (begin + first, begin + first + rot // 2)
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _held64(x, fmt):
    """The 8-bit value nearest to x (ties to even, saturating): steps of 2^(exponent - mantissa bits), exponents not below the least normal one."""
    bits, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    step = torch.exp2((torch.frexp(x)[1].double() - 1).clamp(min=least) - bits)
    return (torch.round(x / step) * step).clamp(-FP8[fmt][1], FP8[fmt][1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {m: _turned64(s[m].reshape(case["tokens"], h, case["d"]), s["positions"], s["inv_freq"], case["rot_begin"],
                             case["rot"], case["interleaved"], case["grad"]) for m, h in (("q", case["hq"]), ("k", case["hk"]))}
    n, lens = _counts(case)
    pt = s["page_table"].cpu().numpy()
    page, hkv, d, fmt = case["page"], case["hkv"], case["d"], case["fmt"]
    rows = [torch.from_numpy(pt[b][np.arange(l) // page].astype(np.int64) * page + np.arange(l) % page).to(DEV) for b, l in enumerate(lens)]
    stored = [(s[m] if fmt == "bf16" else s[m].view(FP8[fmt][0])).view(-1, hkv, d) for m in ("kc", "vc")]
    if case["op"] == "write":
        k = s["k"].reshape(-1, hkv, d)
        k = _turned64(k, s["positions"], s["inv_freq"], 0, case["rot"], case["interleaved"], False) if case["rot"] else k.double()
        v = s["v"].reshape(-1, hkv, d).double()
        out = [x.double() for x in stored]
        new = torch.cat([r[l - m:] for r, m, l in zip(rows, n, lens)])
        for o, x, descale in zip(out, (k, v), (s["kds"], s["vds"])):
            o[new] = x if fmt == "bf16" else _held64(x / descale, fmt)
        return {"k_cache": out[0].view(s["kc"].shape), "v_cache": out[1].view(s["vc"].shape)}
    def of(x, r, descale):
        return x.view(torch.uint8 if fmt != "bf16" else torch.bfloat16)[r].view(x.dtype).double() * descale
    if case["op"] == "read":
        return {m: torch.cat([of(x, r[l - c:], ds) for r, c, l in zip(rows, n, lens)])
                for m, x, ds in (("k", stored[0], s["kds"]), ("v", stored[1], s["vds"]))}
    if float((n * lens).sum()) * case["hq"] * d * 4 > 2e12:
        return None
    o = torch.empty((s["T"], case["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["T"], case["hq"]), dtype=torch.float64, device=DEV)
    g = case["hq"] // hkv
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint64)
    at = 0
    for r, m, l in zip(rows, n, lens):
        m, l = int(m), int(l)
        seen = np.ones((m, l), dtype=bool)
        for i in range(m):
            for j in range(m):
                seen[i, l - m + j] = j <= i if mask is None else bool((int(mask[at + i, j // 64]) >> (j % 64)) & 1)
        seen = torch.from_numpy(seen).to(DEV).repeat_interleave(g, 0)
        for h in range(hkv):
            K, V = (of(x[:, h].contiguous(), r, ds) for x, ds in ((stored[0], s["kds"]), (stored[1], s["vds"])))
            q = s["q"][at:at + m, h * g:(h + 1) * g].double().reshape(m * g, d)
            e = (q @ K.T / math.sqrt(d)).masked_fill(~seen, float("-inf"))
            z = torch.logsumexp(e, 1)
            o[at:at + m, h * g:(h + 1) * g] = ((e - z[:, None]).exp() @ V).view(m, g, d)
            lse[at:at + m, h * g:(h + 1) * g] = z.view(m, g)
        at += m
    return {"o": o, "lse": lse}
