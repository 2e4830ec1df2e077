"""Measured operators: norms of queries and keys with the position rotation in the same pass and their
gradient, attention weight accumulated per cached token, and eviction from a paged cache by it.
``own`` selects the library's calls or the plain form."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases

def _norm(name, tokens, hq, hk, d, rot_begin, rot, interleaved=False, grad=False, f32=False, fused=True, weights=True,
          amplitude=1.0, far=32768):
    return {"name": name, "op": "norm", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot_begin": rot_begin, "rot": rot,
            "interleaved": interleaved, "grad": grad, "f32": f32, "fused": fused, "weights": weights,
            "amplitude": amplitude, "far": far}


def _score(name, B, n_lo, n_hi, lo, hi, hq, hkv, d, page, fmt, decay=1.0, whole=False, lens=1):
    """n queries per sequence, U[n_lo, n_hi], after U[lo, hi] cached tokens; whole: every token of a prompt is one."""
    return {"name": name, "op": "score", "B": B, "n_lo": n_lo, "n_hi": n_hi, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "fmt": fmt, "decay": decay, "whole": whole, "lens": lens}


def _evict(name, B, lo, hi, budget, sinks, recent, hkv, d, page, fmt, lens=1):
    """U[lo, hi] cached tokens of each sequence, of which `budget` stay."""
    return {"name": name, "op": "evict", "B": B, "lo": lo, "hi": hi, "budget": budget, "sinks": sinks, "recent": recent,
            "hkv": hkv, "d": d, "page": page, "fmt": fmt, "lens": lens}


def listed():
    return [
        # one decode step of a batch of 64: q and k of one token each, read out of the fused projection
        _norm("norm_step", 64, 32, 8, 128, 0, 128),
        # packed prefill of eight prompts
        _norm("norm_prefill", 18432, 32, 8, 128, 0, 128),
        # training: gradients of the projection's rows and of both weights
        _norm("norm_grad", 16384, 32, 8, 128, 0, 128, grad=True),
        # training in fp32, the last third of 192-wide heads rotated
        _norm("norm_grad_part", 8192, 16, 16, 192, 128, 64, interleaved=True, grad=True, f32=True, fused=False),
        # one decode step of a batch over long ragged contexts: the new token's weights added to the sums
        _score("score_step", 64, 1, 1, 1024, 32768, 32, 8, 128, 16, "bf16"),
        # the same over an 8-bit cache
        _score("score_step_e4m3", 64, 1, 1, 1024, 32768, 32, 8, 128, 16, "e4m3"),
        # the last 32 tokens of long prompts vote on what is kept of them
        _score("score_window", 16, 32, 32, 2048, 16384, 32, 8, 128, 16, "bf16", decay=0.0),
        # sums over whole prompts
        _score("score_prompt", 8, 0, 0, 512, 4096, 32, 8, 128, 16, "bf16", decay=0.0, whole=True),
        # a few accepted tokens of ragged count, narrow heads, odd pages, older weight faded
        _score("score_ragged", 48, 1, 6, 1, 8000, 12, 3, 64, 7, "e5m2", decay=0.9),
        # one user's short context cut down: latency
        _evict("evict_one", 1, 1000, 1000, 256, 4, 32, 8, 128, 16, "bf16"),
        # prompts cut down to a fixed budget before the decode
        _evict("evict_prompt", 16, 2048, 32768, 2048, 4, 32, 8, 128, 16, "bf16"),
        # during the decode, when sequences have outgrown the budget by some pages
        _evict("evict_step", 64, 4100, 4352, 4096, 4, 256, 8, 128, 16, "e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "score", "score", "evict"])
    seed = rng.randrange(1 << 20)
    if op == "norm":
        d = rng.choice([64, 96, 128, 192, 256])
        half = rng.choice([d // 2, d // 4, 24, 16])
        rot = 2 * half
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 3, 4, 8])
        f32 = rng.random() < 0.3
        grad = rng.random() < 0.5
        most = min(24000, 18432 * 40 * 128 // ((hq + hk) * d * (2 if f32 else 1)))
        c = _norm(None, _log(rng, 1, most), hq, hk, d, rng.choice([0, d - rot]), rot, rng.random() < 0.4, grad, f32,
                  rng.random() < 0.6, rng.random() < 0.8, rng.choice([1.0, 1.0, 1.2]), rng.choice([4096, 32768, 1000000]))
    elif op == "score":
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 3, 4, 8])
        page = rng.choice([1, 7, 16, 16, 64, 256])
        fmt = rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
        decay = rng.choice([0.0, 0.9, 1.0, 1.0])
        B = _log(rng, 1, 64)
        if rng.random() < 0.3:
            # no more scores than the listed prompts
            hi = _log(rng, 1, max(1, min(4096, int(math.sqrt(8 * 2304**2 * 32 / (B * hkv * g))))))
            c = _score(None, B, 0, 0, rng.choice([1, hi]), hi, hkv * g, hkv, d, page, fmt, decay, True, seed)
        else:
            n_hi = _log(rng, 1, 96)
            n_lo = rng.choice([1, n_hi])
            hi = _log(rng, 1, max(1, min(32768, 16 * 16384 * 32 * 32 // (B * hkv * g * n_hi), 64 * 32768 // B)))
            c = _score(None, B, n_lo, n_hi, rng.choice([1, hi, max(1, hi // 32)]), hi, hkv * g, hkv, d, page, fmt, decay, False, seed)
    else:
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 5, 8])
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(32768, 500000 // B))
        budget = _log(rng, 1, hi)
        sinks = rng.choice([0, min(4, budget)])
        recent = rng.randint(0, budget - sinks)
        c = _evict(None, B, rng.choice([1, hi, max(1, hi // 8)]), hi, budget, sinks, recent, hkv, d,
                   rng.choice([1, 7, 16, 16, 64, 256]), rng.choice(["bf16", "bf16", "e4m3", "e5m2"]), seed)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ shapes

def _counts(case):
    """(queries, cached tokens with theirs) of each sequence; the same for every seed."""
    rs = np.random.RandomState(case["lens"])
    B = case["B"]
    lens = rs.randint(case["lo"], case["hi"] + 1, B)
    if case["op"] == "evict":
        return np.zeros(B, dtype=lens.dtype), lens
    n = lens if case["whole"] else rs.randint(case["n_lo"], case["n_hi"] + 1, B)
    return n, (lens if case["whole"] else lens + n)


def _elem(case):
    return 2 if case["fmt"] == "bf16" else 1


def work(case):
    if case["op"] == "norm":
        e, n = 4 if case["f32"] else 2, case["tokens"] * (case["hq"] + case["hk"])
        fixed = 4 * case["tokens"] + 4 * case["rot"]
        w = 8 * case["d"] if case["weights"] else 0
        if case["grad"]:
            return {"bytes": 3 * n * case["d"] * e + fixed + 2 * w, "flops": n * (3 * case["rot"] + 12 * case["d"])}
        return {"bytes": 2 * n * case["d"] * e + fixed + w, "flops": n * (3 * case["rot"] + 4 * case["d"])}
    n, lens = _counts(case)
    hkv, d, e = case["hkv"], case["d"], _elem(case)
    pages = -(-lens // case["page"])
    table = 4 * int(pages.sum()) + 4 * len(lens)
    if case["op"] == "score":
        seen = int((n * lens - n * (n - 1) // 2).sum())  # query i of n does not see the n - 1 - i tokens after its own
        sums = 4 * hkv * int((2 * lens - n if case["decay"] else lens).sum())
        return {"bytes": int(lens.sum()) * hkv * d * e + sums + int(n.sum()) * case["hq"] * (2 * d + 4) + table,
                "flops": 2 * seen * case["hq"] * d}
    # sequences above the budget are looked through; the last tokens move, and of those chosen between them and the first
    # ones, by their number, the share that lies behind the slots for it
    K, edge = case["budget"], case["sinks"] + case["recent"]
    long = lens[lens > K]
    rows = hkv * float((case["recent"] + (K - edge) * (long - K) / np.maximum(long - edge, 1)).sum())
    return {"bytes": 4 * int(long.sum()) * hkv + 4 * len(lens) * hkv * K + int(2 * rows * (2 * d * e + 4)) + table,
            "flops": int(long.sum()) * hkv}


# ------------------------------------------------------------------------------------ inputs

def _inv_freq(rot, dev):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)


def _pages(case, lens, rs):
    """Page table of a pool that a seeded permutation hands out, with some pages that no sequence holds."""
    pages = -(-lens // case["page"])
    num = int(pages.sum()) + 3
    perm = rs.permutation(num).astype(np.int32)
    ends = np.cumsum(pages)
    pt = np.full((len(lens), int(pages.max())), -1, dtype=np.int32)
    for b in range(len(lens)):
        pt[b, :pages[b]] = perm[ends[b] - pages[b]:ends[b]]
    return pt, num


def _cache(case, num, g):
    """A cache of values N(0, 1) (8-bit: codes of x / descale) and its descale."""
    x = torch.randn((num, case["page"], case["hkv"], case["d"]), generator=g, device=DEV, dtype=torch.bfloat16)
    if case["fmt"] == "bf16":
        return x, 1.0
    t, big = FP8[case["fmt"]]
    x = (x.float() * (big / 6.0)).clamp(-big, big).to(t).view(torch.uint8)
    return x, float(np.float32(6.0 / big))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}
    if case["op"] == "norm":
        T, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        t = torch.float32 if case["f32"] else torch.bfloat16
        if case["fused"]:  # q, k and v side by side, as the projection leaves them; the gradients go where it reads them
            x, y = (torch.randn((T, (hq + 2 * hk) * d), generator=g, device=DEV, dtype=t) for _ in range(2))
            s["q"], s["k"] = x[:, :hq * d], x[:, hq * d:(hq + hk) * d]
            if case["grad"]:
                s["dq"], s["dk"] = y[:, :hq * d], y[:, hq * d:(hq + hk) * d]
        else:
            s["q"], s["k"] = (torch.randn((T, h * d), generator=g, device=DEV, dtype=t) for h in (hq, hk))
            if case["grad"]:
                s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["wq"], s["wk"] = ((1 + 0.3 * torch.randn(d, generator=g, device=DEV)) if case["weights"] else None for _ in range(2))
        if case["grad"]:
            s["dq_out"], s["dk_out"] = (torch.randn((T, h, d), generator=g, device=DEV, dtype=t) for h in (hq, hk))
            s["dwq"], s["dwk"] = (torch.empty(d, device=DEV) if case["weights"] else None for _ in range(2))
        else:
            s["q_out"], s["k_out"] = (torch.empty((T, h, d), dtype=t, device=DEV) for h in (hq, hk))
        s["positions"] = torch.from_numpy(rs.randint(0, case["far"], T).astype(np.int32)).to(DEV)
        s["inv_freq"] = _inv_freq(case["rot"], DEV)
        return s
    n, lens = _counts(case)
    pt, num = _pages(case, lens, rs)
    B, hkv, d = case["B"], case["hkv"], case["d"]
    s.update(B=B, num=num, width=pt.shape[1], T=int(n.sum()), max_q=int(n.max()), longest=int(lens.max()))
    s["page_table"] = torch.from_numpy(pt).to(DEV)
    s["seqlens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
    s["kc"], s["kds"] = _cache(case, num, g)
    if case["op"] == "evict":
        s["vc"], _ = _cache(case, num, g)
        # heavy-tailed sums, some tokens never looked at
        x = torch.randn((num, hkv, case["page"]), generator=g, device=DEV)
        s["score"] = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.1, 0.0, torch.exp(2 * x))
        s["kept"] = torch.empty((B, hkv, case["budget"]), dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
        return s
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    s["dense"] = bool((n == n[0]).all())  # equal counts: no offsets needed
    s["score"] = torch.rand((num, hkv, case["page"]), generator=g, device=DEV)
    s["q"] = torch.randn((s["T"], case["hq"], d), generator=g, device=DEV, dtype=torch.bfloat16) * 2
    s["lse"] = _row_lse(s)
    return s


# ------------------------------------------------------------------------------------ plain form

def _rotated(x, angle, begin, rot, interleaved, amplitude, back=False):
    """x [T, H, d] in 32 bits; back: the gradient."""
    c, sn = (amplitude * angle.cos()).float()[:, None], (amplitude * angle.sin()).float()[:, None]
    if back:
        sn = -sn
    part = x[..., begin:begin + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((x[..., :begin], turned, x[..., begin + rot:]), -1)


def _normed(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # 64 bits: far positions
    place = (angle, c["rot_begin"], c["rot"], c["interleaved"], c["amplitude"])
    out = {}
    for m, h in (("q", c["hq"]), ("k", c["hk"])):
        x, w = s[m].reshape(c["tokens"], h, c["d"]).float(), s["w" + m]
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        if not c["grad"]:
            y = x * r if w is None else x * r * w
            out[m] = _rotated(y, *place).to(s[m].dtype)
            continue
        g = _rotated(s[f"d{m}_out"].float(), *place, back=True)
        xn = x * r
        gw = g if w is None else g * w
        dx = r * (gw - xn * (xn * gw).mean(-1, keepdim=True))
        s["d" + m].copy_(dx.view(c["tokens"], -1))
        out["d" + m] = s["d" + m]
        if w is not None:
            out["dw" + m] = (xn * g).sum((0, 1), dtype=torch.float64).float()
    return out


def _keys(s):
    """[B, hkv, width * page, d] in 32 bits, zeros where a sequence holds nothing."""
    c = s["case"]
    L = s["width"] * c["page"]
    x = s["kc"][s["page_table"].clamp(min=0)].view(s["B"], L, c["hkv"], c["d"])
    x = x.float() if c["fmt"] == "bf16" else x.view(FP8[c["fmt"]][0]).float() * s["kds"]
    held = torch.arange(L, device=DEV) < s["seqlens"].long()[:, None]
    return torch.where(held[..., None, None], x, 0.0).transpose(1, 2)


def _logits(s):
    """(scaled scores [B, hkv, n * G, L] of a batch padded to the longest, -inf where a query does not see the token;
    sequence and index of every packed row)."""
    c = s["case"]
    B, hkv, n, G, L = s["B"], c["hkv"], s["max_q"], c["hq"] // c["hkv"], s["width"] * c["page"]
    cu, t = s["cu"].long(), torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    q = torch.zeros((B, n, hkv, G, c["d"]), device=DEV)
    q[b, i] = s["q"].float().view(-1, hkv, G, c["d"])
    score = q.permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, c["d"]) @ _keys(s).transpose(2, 3)
    score.mul_(1.0 / math.sqrt(c["d"]))
    count = cu[1:] - cu[:-1]
    last = (s["seqlens"].long() - count)[:, None] + torch.arange(n, device=DEV)  # the last token that query i sees
    last = torch.where(torch.arange(n, device=DEV) < count[:, None], last, -1)
    unseen = torch.arange(L, device=DEV) > last[..., None]
    score.view(B, hkv, n, G, L).masked_fill_(unseen[:, None, :, None], float("-inf"))
    return score, b, i


def _row_lse(s):
    """log of the sum of exponentials of every row's scores, [T, hq], as the attention call returned it."""
    c = s["case"]
    score, b, i = _logits(s)
    lse = score.logsumexp(-1).view(s["B"], c["hkv"], s["max_q"], -1).permute(0, 2, 1, 3)
    return lse[b, i].reshape(s["T"], c["hq"])


def _scored(s):
    c = s["case"]
    score, b, i = _logits(s)
    lse = torch.zeros((s["B"], s["max_q"], c["hkv"], c["hq"] // c["hkv"]), device=DEV)
    lse[b, i] = s["lse"].view(-1, c["hkv"], c["hq"] // c["hkv"])
    total = score.sub_(lse.permute(0, 2, 1, 3).reshape(s["B"], c["hkv"], -1, 1)).exp_().sum(2)
    at = torch.nonzero(torch.arange(total.shape[2], device=DEV) < s["seqlens"].long()[:, None])
    page, slot = s["page_table"][at[:, 0], at[:, 1] // c["page"]].long(), at[:, 1] % c["page"]
    new = total[at[:, 0], :, at[:, 1]]
    if c["decay"]:  # the queries' own tokens are new: what their slots hold is of no token
        old = at[:, 1] < (s["seqlens"] - (s["cu"][1:] - s["cu"][:-1]))[at[:, 0]]
        new = new + torch.where(old[:, None], c["decay"] * s["score"][page, :, slot], 0.0)
    s["score"][page, :, slot] = new
    return {"score": s["score"]}


def _as_values(x, fmt):
    return x if fmt == "bf16" else x.view(FP8[fmt][0])


def _evicted(s):
    c = s["case"]
    page, hkv, K, L = c["page"], c["hkv"], c["budget"], s["width"] * c["page"]
    lens = s["seqlens"].long()
    t = torch.arange(L, device=DEV)
    gone = lens > K  # the others keep all they have
    rank = s["score"][s["page_table"].clamp(min=0)].permute(0, 2, 1, 3).reshape(s["B"], hkv, L)
    always = (t < c["sinks"]) | (t >= lens[:, None] - c["recent"])
    rank = torch.where(always[:, None], float("inf"), rank).masked_fill_((t >= lens[:, None])[:, None], float("-inf"))
    order = rank.sort(dim=-1, descending=True, stable=True)[1][..., :K]  # ties: the earlier token
    stays = torch.zeros(rank.shape, dtype=torch.bool, device=DEV).scatter_(2, order, True) & gone[:, None, None]
    # a kept token stays in its slot if that is left; the last ones close up, the others fill the holes in turn
    j, end = torch.arange(K, device=DEV), K - c["recent"]
    new = lens.clamp(max=K)
    kept = torch.where(gone[:, None] & (j >= end), j + lens[:, None] - K, torch.where(j < new[:, None], j, -1))
    kept = kept[:, None].expand(-1, hkv, -1).clone()
    hole = torch.zeros_like(kept, dtype=torch.bool)
    hole[..., :L] = ~stays[..., :K] & ((j < end)[:L] & gone[:, None])[:, None]
    tail = stays & ((t >= end) & (t < lens[:, None] - c["recent"]))[:, None]
    kept[hole] = torch.nonzero(tail)[:, 2]
    s["kept"].copy_(kept)
    s["new_lens"].copy_(new)
    b, h, j = torch.nonzero(kept > j).unbind(1)
    src = kept[b, h, j]
    sp, ss = s["page_table"][b, src // page].long(), src % page
    dp, ds = s["page_table"][b, j // page].long(), j % page
    for x in (s["kc"], s["vc"]):
        x[dp, ds, h] = x[sp, ss, h]
    s["score"][dp, h, ds] = s["score"][sp, h, ss]
    return _state(s)


def _state(s):
    fmt = s["case"]["fmt"]
    return {"kept": s["kept"], "new_lens": s["new_lens"], "k_cache": _as_values(s["kc"], fmt),
            "v_cache": _as_values(s["vc"], fmt), "score": s["score"]}


# ------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"norm": _normed, "score": _scored, "evict": _evicted}[s["case"]["op"]](s)


def _run_own(s):
    import exact_softmax_attention_gb300 as A

    c = s["case"]
    if c["op"] == "norm":
        t = "f32" if c["f32"] else "bf16"
        T, hq, hk, d = c["tokens"], c["hq"], c["hk"], c["d"]
        if not c["grad"]:
            A.attn_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["wq"], s["wk"], EPS, s["positions"], s["inv_freq"], T,
                                hq, hk, d, c["rot_begin"], c["rot"], s["q"].stride(0), s["k"].stride(0), hq * d, hk * d, t,
                                c["interleaved"], c["amplitude"])
            return {"q": s["q_out"], "k": s["k_out"]}
        A.attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["wq"], s["wk"], EPS, s["positions"], s["inv_freq"],
                                s["dq"], s["dk"], s["dwq"], s["dwk"], T, hq, hk, d, c["rot_begin"], c["rot"], s["q"].stride(0),
                                s["k"].stride(0), hq * d, hk * d, s["dq"].stride(0), s["dk"].stride(0), t, c["interleaved"],
                                c["amplitude"])
        out = {"dq": s["dq"], "dk": s["dk"]}
        if c["weights"]:
            out.update(dwq=s["dwq"], dwk=s["dwk"])
        return out
    if c["op"] == "score":
        A.attn_kv_score_paged(s["q"], s["lse"], s["kc"], s["score"], s["page_table"], s["seqlens"], None if s["dense"] else s["cu"],
                              c["page"], s["T"], s["B"], s["max_q"], c["hq"], c["hkv"], c["d"], s["width"], s["num"],
                              1.0 / math.sqrt(c["d"]), c["decay"], c["fmt"], s["kds"])
        return {"score": s["score"]}
    A.attn_kv_select_paged(s["score"], s["page_table"], s["seqlens"], s["kept"], s["new_lens"], c["page"], s["B"], c["hkv"],
                           s["width"], s["num"], c["budget"], c["sinks"], c["recent"])
    A.attn_kv_compact_paged(s["kc"], s["vc"], s["score"], s["kept"], s["new_lens"], s["page_table"], c["page"], s["B"], c["hkv"],
                            c["d"], s["width"], s["num"], c["budget"], c["fmt"])
    return _state(s)


# ------------------------------------------------------------------------------------ 64 bits

def _turned64(x, angle, c):
    """The rotation pair by pair as complex numbers: x [T, H, d]."""
    turn = torch.polar(torch.full_like(angle, c["amplitude"]), angle).unsqueeze(1)
    first = torch.arange(c["rot"] // 2, device=x.device)
    if c["interleaved"]:
        a, b = c["rot_begin"] + 2 * first, c["rot_begin"] + 2 * first + 1
    else:
        a, b = c["rot_begin"] + first, c["rot_begin"] + first + c["rot"] // 2
    z = torch.complex(x[..., a], x[..., b]) * turn
    return x.index_copy(-1, a, z.real).index_copy(-1, b, z.imag)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        angle = s["positions"].double().unsqueeze(1).mul(s["inv_freq"])
        out = {}
        for m, h in (("q", case["hq"]), ("k", case["hk"])):
            x = s[m].reshape(case["tokens"], h, case["d"]).double()
            w = torch.ones(case["d"], dtype=torch.float64, device=DEV) if s["w" + m] is None else s["w" + m].double()
            with torch.enable_grad():
                x.requires_grad_(case["grad"])
                w.requires_grad_(case["grad"])
                y = _turned64(x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w, angle, case)
                if not case["grad"]:
                    out[m] = y
                    continue
                dx, dw = torch.autograd.grad(y, (x, w), s[f"d{m}_out"].double())
            out["d" + m] = dx.reshape(case["tokens"], -1)
            if s["w" + m] is not None:
                out["dw" + m] = dw
        return out
    n, lens = _counts(case)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    pt = s["page_table"].cpu().numpy()
    if case["op"] == "score":
        G, at = case["hq"] // hkv, 0
        sums = s["score"].double()
        for b in range(case["B"]):
            m, l = int(n[b]), int(lens[b])
            where = torch.from_numpy(pt[b][np.arange(l) // page].astype(np.int64)).to(DEV), torch.arange(l, device=DEV) % page
            hidden = torch.arange(l, device=DEV)[None] > torch.arange(l - m, l, device=DEV)[:, None]
            for h in range(hkv):
                K = s["kc"][where[0], where[1], h]
                K = K.double() if case["fmt"] == "bf16" else K.view(FP8[case["fmt"]][0]).double() * s["kds"]
                new = torch.zeros(l, dtype=torch.float64, device=DEV)
                for r in range(h * G, (h + 1) * G):
                    e = s["q"][at:at + m, r].double() @ K.T / math.sqrt(d) - s["lse"][at:at + m, r].double()[:, None]
                    new += e.exp().masked_fill(hidden, 0.0).sum(0)
                new[:l - m] += sums[where[0], h, where[1]][:l - m] * case["decay"]
                sums[where[0], h, where[1]] = new
            at += m
        return {"score": sums}
    score, kc, vc = s["score"].cpu().numpy(), s["kc"].clone(), s["vc"].clone()
    moved = s["score"].clone()
    kept = np.full((case["B"], hkv, case["budget"]), -1, dtype=np.int32)
    for b in range(case["B"]):
        l = int(lens[b])
        k = min(l, case["budget"])
        tok = np.arange(l)
        where = pt[b][tok // page]
        at = torch.from_numpy(where.astype(np.int64)).to(DEV), torch.from_numpy(tok % page).to(DEV)
        for h in range(hkv):
            kept[b, h, :k] = tok[:k]
            if l > k:
                first, end = case["sinks"], k - case["recent"]
                middle = tok[first:l - case["recent"]]
                best = set(middle[np.lexsort((middle, -score[where, h, tok % page][middle]))][:end - first].tolist())
                behind = iter(sorted(x for x in best if x >= end))
                kept[b, h, first:end] = [x if x in best else next(behind) for x in range(first, end)]
                kept[b, h, end:] = tok[l - case["recent"]:]
            src, dst = torch.from_numpy(kept[b, h, :k]).to(DEV).long(), torch.arange(k, device=DEV)
            for new, old in ((kc, s["kc"]), (vc, s["vc"])):
                new[at[0][dst], at[1][dst], h] = old[at[0][src], at[1][src], h]
            moved[at[0][dst], h, at[1][dst]] = s["score"][at[0][src], h, at[1][src]]
    return {"kept": torch.from_numpy(kept).to(DEV), "new_lens": torch.from_numpy(np.minimum(lens, case["budget"]).astype(np.int32)).to(DEV),
            "k_cache": _as_values(kc, case["fmt"]), "v_cache": _as_values(vc, case["fmt"]), "score": moved}
