"""What the operators of a compressed paged cache are measured on.

A cache that outgrows its pages is made smaller in two ways: its keys and values are held in 8
bits (E4M3) with a power-of-two scale for each page and head, and the keys that the queries give
little weight are taken out of it.  Four of the library's operators do that: the new rows enter
8-bit pages (dllm_paged_append_f8), the queries attend over them (dllm_paged_attention_f8), every
key's attention weight is added to its score (dllm_paged_weights), and the slots of the lowest
scores are given to later keys that stay (dllm_paged_evict).  Each case is one pass through one.

Where `own` is false, `run` computes the operators in their plain form (elementary torch
operations); where it is true, it makes the library's calls on the same state.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
E_MIN, E_MAX = -64, 63          # exponents that a page's scale takes
MAX_CODE = 448.0                # the largest E4M3 value


# ---------------------------------------------------------------------------- the cases
def _append(name, B, new, kv, ragged, n_q, n_kv, hd, page, src, norm, pad=0):
    return {"name": name, "op": "append", "B": B, "new": new, "kv": kv, "ragged": ragged, "n_q": n_q, "n_kv": n_kv,
            "hd": hd, "page": page, "src": src, "dtype": "f8", "norm": norm, "pad": pad}


def _attend(name, B, new, kv, ragged, n_q, n_kv, hd, page, mask, pad=0):
    return {"name": name, "op": "attend", "B": B, "new": new, "kv": kv, "ragged": ragged, "n_q": n_q, "n_kv": n_kv,
            "hd": hd, "page": page, "dtype": "f8", "mask": mask, "pad": pad}


def _weigh(name, B, new, kv, ragged, n_q, n_kv, hd, page, dtype, mask, pad=0):
    return {"name": name, "op": "weigh", "B": B, "new": new, "kv": kv, "ragged": ragged, "n_q": n_q, "n_kv": n_kv,
            "hd": hd, "page": page, "dtype": dtype, "mask": mask, "pad": pad}


def _evict(name, B, kv, keep, ragged, n_kv, hd, page, dtype, recent):
    return {"name": name, "op": "evict", "B": B, "new": 1, "kv": kv, "keep": keep, "ragged": ragged, "n_kv": n_kv,
            "hd": hd, "page": page, "dtype": dtype, "recent": recent, "pad": 0}


def listed():
    return [
        # the current block of one LLaDA-8B-shaped sequence enters pages that are half full (latency)
        _append("append8_block", 1, 32, 1024, 0, 32, 32, 128, 64, "bf16", False),
        # four ragged prompts, normed heads, the whole fused projection output, padded batch
        _append("append8_prompts", 4, 2048, 2048, 30, 32, 32, 128, 64, "bf16", True, 96),
        # a block of masked tokens of one LLaDA-8B-shaped sequence over its cache (latency)
        _attend("attend8_block", 1, 32, 1024, 0, 32, 32, 128, 64, 0),
        # single tokens of 64 ragged sequences, grouped heads, small pages
        _attend("attend8_tokens", 64, 1, 8192, 50, 28, 4, 128, 16, 1, 3),
        # blocks of 16 ragged sequences, one query head per key head
        _attend("attend8_blocks", 16, 32, 4096, 50, 32, 32, 128, 64, 0),
        # the second half of two long prompts, blocks of 32 see the blocks up to their own
        _attend("attend8_prompts", 2, 4096, 8192, 10, 28, 4, 128, 128, 32),
        # the weights that 64 ragged sequences' tokens give their keys, 8-bit cache
        _weigh("weigh_tokens", 64, 1, 8192, 50, 28, 4, 128, 16, "f8", 1, 3),
        # the same of blocks of 16 ragged sequences over a bf16 cache
        _weigh("weigh_blocks", 16, 32, 4096, 50, 32, 32, 128, 64, "bf16", 0),
        # the tiny fp32 layer's heads over an odd-sized cache
        _weigh("weigh_f32", 4, 32, 2001, 20, 8, 8, 64, 32, "f32", 1),
        # one LLaDA-8B-shaped sequence gives up as many keys as its last block brought (latency)
        _evict("evict_block", 1, 1056, 1024, 0, 32, 128, 64, "bf16", 32),
        # 64 ragged sequences fall to three quarters, 8-bit cache, small pages
        _evict("evict_requests", 64, 8192, 6144, 50, 4, 128, 16, "f8", 256),
        # 16 sequences fall to half, one key head per query head
        _evict("evict_half", 16, 4096, 2048, 20, 32, 128, 64, "bf16", 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weigh", "evict"])
    n_q, n_kv, hd = rng.choice([(32, 32, 128), (28, 4, 128), (8, 8, 64), (16, 2, 128), (12, 4, 64), (8, 1, 128)])
    page = rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 64)
    ragged = rng.choice([0, 20, 50])
    if op == "append":
        new = _log(rng, 1, max(1, 6000 // B))
        kv = new + rng.choice([0, _log(rng, 1, 8192)])
        return _append(None, B, new, kv, ragged, n_q, n_kv, hd, page, rng.choice(["bf16", "bf16", "f32"]),
                       rng.random() < 0.5, rng.choice([0, 0, 7]))
    if op == "evict":
        kv = _log(rng, 40, max(41, min(65536, 64 * 8192 * 4 // (B * n_kv))))
        keep = max(1, kv * rng.choice([50, 75, 90, 97]) // 100)
        return _evict(None, B, kv, keep, ragged, n_kv, hd, page, rng.choice(["bf16", "f8", "f8", "f32"]),
                      rng.choice([0, 16, min(64, keep)]))
    dtype = "f8" if op == "attend" else rng.choice(["f8", "f8", "bf16", "bf16", "f32"])
    new = rng.choice([1, _log(rng, 2, 40), _log(rng, 8, 4096)])
    most = 2 * 4096 * 8192 * 28 * 128 // (B * new * n_q * hd)
    most = min(most, 64 * 8192 * 4 // (B * n_kv), 65536)
    if dtype == "f32":
        most = min(most // 64, 4096)
        new = min(new, 64)
    if op == "weigh":
        new = min(new, 512)
    kv = max(new, _log(rng, 16, max(17, most)))
    if op == "attend":
        return _attend(None, B, new, kv, ragged, n_q, n_kv, hd, page, rng.choice([0, 1, 32]), rng.choice([0, 0, 5]))
    return _weigh(None, B, new, kv, ragged, n_q, n_kv, hd, page, dtype, rng.choice([0, 1, 32]), rng.choice([0, 0, 5]))


def _lengths(case):
    """(new rows, keys after them) of each sequence: part of the case, the same for every seed."""
    r = random.Random(977 * case["B"] + 31 * case["new"] + case["kv"])
    cut = case["ragged"] / 100.0
    new = [max(1, case["new"] - int(case["new"] * cut * r.random() * (b > 0))) for b in range(case["B"])]
    kv = [max(n, case["kv"] - int(case["kv"] * cut * r.random() * (b > 0))) for b, n in enumerate(new)]
    return new, kv


def _visible(case, new, kv):
    """Keys that the rows see, summed over all of them."""
    m = case["mask"]
    if m == 0:
        return sum(n * k for n, k in zip(new, kv))
    return sum(min(k, ((k - n + s) // m + 1) * m) for n, k in zip(new, kv) for s in range(n))


def work(case):
    new, kv = _lengths(case)
    hd, n_kv, page = case["hd"], case["n_kv"], case["page"]
    el = {"f8": 1, "bf16": 2, "f32": 4}[case["dtype"]]
    small = 4 * (sum(kv) // page + 3 * case["B"])       # table, starts, lengths
    if case["op"] == "evict":
        keep = case["keep"]
        # (scores without order: of the slots past `keep`, as large a share stays as of all)
        moved = sum(max(0, k - keep) * keep / max(k, 1) for k in kv) * n_kv
        stay = sum(min(k, keep) for k in kv) * n_kv
        return {"bytes": 8 * sum(kv) * n_kv + 8 * stay + 4 * moved * hd * el + small, "flops": 2 * sum(kv) * n_kv}
    n_q = case["n_q"]
    scales = 2 * n_kv * sum(-(-k // page) for k in kv) if case["dtype"] == "f8" else 0
    if case["op"] == "append":
        src = 2 if case["src"] == "bf16" else 4
        return {"bytes": sum(new) * hd * ((n_q + 2 * n_kv) * src + n_q * 2 + 2 * n_kv) + small + 4 * hd,
                "flops": sum(new) * (n_q + n_kv) * hd * (7 if case["norm"] else 3) + 2 * sum(new) * n_kv * hd}
    q_el = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "weigh":
        return {"bytes": sum(new) * n_q * (hd * q_el + 4) + sum(kv) * n_kv * (hd * el + 8) + small + scales // 2,
                "flops": 2 * _visible(case, new, kv) * n_q * hd}
    return {"bytes": 2 * sum(new) * n_q * hd * 2 + 2 * sum(kv) * n_kv * hd + small + scales,
            "flops": 4 * _visible(case, new, kv) * n_q * hd}


# ---------------------------------------------------------------------------- inputs
def _codes(x):
    """x [n_pages, page, n_kv, hd] fp32 -> (E4M3 codes, E8M0 scales [n_pages, n_kv])."""
    e = _needed(x.abs().amax((1, 3)))
    q = (x * torch.exp2(-e.float())[:, None, :, None]).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=dev, dtype=torch.float32)

    s = {"case": case}
    new, kv = _lengths(case)
    hd, n_kv, page, B = case["hd"], case["n_kv"], case["page"], case["B"]
    f8 = case["dtype"] == "f8"
    dt = DT[case["dtype"]]
    qdt = torch.bfloat16 if f8 else dt
    need = [-(-k // page) for k in kv]
    P = sum(need) + 2
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    s["table"] = table.to(dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32).to(dev)
    s["K_scale"] = s["V_scale"] = None
    # (channels of unlike size, as keys have after the rotation)
    loud = torch.exp(0.5 * randn(n_kv, hd))
    s["K_pages"], s["V_pages"] = randn(P, page, n_kv, hd) * loud / loud.square().mean(-1, keepdim=True).sqrt(), randn(P, page, n_kv, hd)
    if f8:
        (s["K_pages"], s["K_scale"]), (s["V_pages"], s["V_scale"]) = _codes(s["K_pages"]), _codes(s["V_pages"])
    else:
        s["K_pages"], s["V_pages"] = s["K_pages"].to(dt), s["V_pages"].to(dt)
    slots = max(need) * page
    if case["op"] in ("weigh", "evict"):
        # what eight earlier steps have added up, and the position of each slot's token
        each = 8.0 * case.get("n_q", n_kv) / n_kv * case["new"] / case["kv"]
        s["score"] = torch.rand((B, n_kv, slots), generator=g, device=dev).square_() * (3 * each)
        s["pos_base"] = torch.randint(0, 1000, (B,), generator=g, device=dev, dtype=torch.int32)
        s["slot_pos"] = (torch.arange(slots, dtype=torch.int32, device=dev) + s["pos_base"][:, None])[:, None].repeat(1, n_kv, 1)
    if case["op"] == "evict":
        s["keep"] = torch.full((B,), case["keep"], dtype=torch.int32, device=dev)
        s["out"] = (torch.zeros_like(s["score"]), torch.zeros_like(s["slot_pos"]), torch.zeros_like(s["kv_len"]),
                    torch.zeros_like(s["pos_base"]))
        return s
    n_q = case["n_q"]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    T = sum(new) + case["pad"]
    s["q_start"] = torch.tensor(starts, dtype=torch.int32).to(dev)
    s["max_new"], s["rows"] = max(new), sum(new)
    if case["op"] == "append":
        qkv = randn(T, n_q + 2 * n_kv, hd).to(DT[case["src"]])   # the fused projection's output
        s["Q"], s["K"], s["V"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        s["out"] = torch.zeros((T, n_q, hd), device=dev, dtype=qdt)
        s["gq"] = s["gk"] = None
        if case["norm"]:
            s["gq"] = (1 + 0.1 * randn(hd)).to(qdt)
            s["gk"] = (1 + 0.1 * randn(hd)).to(qdt)
        s["inv_freq"] = (10000.0 ** (-2 * torch.arange(hd // 2, dtype=torch.float64) / hd)).float().to(dev)
        return s
    s["Q"] = (randn(T, n_q, hd) * 1.5).to(qdt)
    if case["op"] == "attend":
        s["out"] = torch.zeros((T, n_q, hd), device=dev, dtype=qdt)
        return s
    s["score_out"] = torch.zeros_like(s["score"])
    # what the attention before it left: each row's log-sum-exp
    s["lse"] = torch.zeros((T, n_q), device=dev)
    at = 0
    for b, (n, k) in enumerate(zip(new, kv)):
        pos = torch.arange(k - n, k, device=dev)
        lim = _limits(pos, torch.full_like(pos, k), case["mask"])
        keys = _values(s, "K", s["table"][b, :need[b]].long()).reshape(-1, n_kv, hd)[:k]
        step = max(1, (1 << 27) // (n_q * k))
        for r in range(0, n, step):
            q = s["Q"][at + r:at + min(n, r + step)].float().view(-1, n_kv, n_q // n_kv, hd)
            sc = torch.einsum("sgjd,lgd->sgjl", q, keys) * (1.0 / math.sqrt(hd))
            dead = torch.arange(k, device=dev)[None, :] >= lim[r:r + step, None]
            sc.masked_fill_(dead[:, None, None, :], float("-inf"))
            s["lse"][at + r:at + min(n, r + step)] = torch.logsumexp(sc, -1).reshape(-1, n_q)
        at += n
    return s


# ---------------------------------------------------------------------------- the plain forms
def _needed(amax):
    """The least exponent e with amax <= 448 * 2^e, within the range a scale takes."""
    m, x = torch.frexp(amax.double())                      # amax = m 2^x, m in [1/2, 1)
    e = torch.where(m <= MAX_CODE / 512, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX).to(torch.int32)


def _exponent(scale):
    return scale.view(torch.uint8).int() - 127


def _values(s, which, pages):
    """The fp32 values of some pages, [..., page, n_kv, hd]."""
    x = s[which + "_pages"][pages].float()
    if s[which + "_scale"] is None:
        return x
    return x * torch.exp2(_exponent(s[which + "_scale"])[pages].float())[..., None, :, None]


def _where(s):
    """Sequence and position of every new row."""
    t = torch.arange(s["rows"], device=s["q_start"].device)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    pos = t - s["q_start"].long()[b] + s["kv_len"].long()[b] - (s["q_start"].long()[b + 1] - s["q_start"].long()[b])
    return b, pos


def _limits(pos, kv_len, m):
    return kv_len if m == 0 else torch.minimum(kv_len, (pos // m + 1) * m)


def _normed(x, gamma, eps):
    if gamma is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.float()


def _rotated(x, cos, sin):
    h = x.shape[-1] // 2
    a, c = x[..., :h], x[..., h:]
    return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)


def _enter(s, which, x, b, pos):
    """Rows x [rows, n_kv, hd] into their pages; a page's scale grows with them and its earlier rows follow."""
    pages, scale = s[which + "_pages"], s[which + "_scale"].view(torch.uint8)
    P, page, n_kv, _ = pages.shape
    pg = s["table"].long()[b, pos // page]
    top = torch.zeros((P, n_kv), device=x.device).scatter_reduce_(0, pg[:, None].expand(-1, n_kv), x.abs().amax(-1), "amax")
    first = torch.full((P,), page, device=x.device).scatter_reduce_(0, pg, pos % page, "amin")   # page: no new row
    need, old = _needed(top) + 127, scale.int()
    now = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
    now = torch.where((first < page)[:, None], now, old)
    grown = ((now > old) & (first > 0)[:, None]).any(1).nonzero()[:, 0]
    kept = torch.arange(page, device=x.device)[None, :] < first[grown, None]
    moved = pages[grown].float() * torch.exp2((old - now)[grown].float())[:, None, :, None]
    bits = pages.view(torch.uint8)
    bits[grown] = torch.where(kept[:, :, None, None], moved.to(pages.dtype).view(torch.uint8), bits[grown])
    bits[pg, pos % page] = (x * torch.exp2(127.0 - now[pg].float())[..., None]).to(pages.dtype).view(torch.uint8)
    scale.copy_(now)


def _plain_append(s):
    b, pos = _where(s)
    ang = pos.double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    n = s["rows"]
    q = _rotated(_normed(s["Q"][:n].float(), s["gq"], 1e-6), cos, sin)
    k = _rotated(_normed(s["K"][:n].float(), s["gk"], 1e-6), cos, sin)
    _enter(s, "K", k, b, pos)
    _enter(s, "V", s["V"][:n].float(), b, pos)
    s["out"][:n] = q.to(s["out"].dtype)
    return s["out"], s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"]


def _padded(s):
    """Queries and limits as [B, max_new, ...], with each row's place."""
    n_kv, hd = s["K_pages"].shape[2:]
    B, n_q = s["table"].shape[0], s["Q"].shape[1]
    b, pos = _where(s)
    slot = torch.arange(s["rows"], device=b.device) - s["q_start"].long()[b]
    q = torch.zeros((B, s["max_new"], n_q, hd), device=b.device)
    q[b, slot] = s["Q"][:s["rows"]].float()
    lim = torch.zeros((B, s["max_new"]), dtype=torch.int64, device=b.device)
    lim[b, slot] = _limits(pos, s["kv_len"].long()[b], s["case"]["mask"])
    return q.view(B, s["max_new"], n_kv, n_q // n_kv, hd), lim, b, slot


def _plain_attend(s):
    n_kv, hd = s["K_pages"].shape[2:]
    B, n_q = s["table"].shape[0], s["Q"].shape[1]
    pages = s["table"].long().clamp(min=0)
    k = _values(s, "K", pages).reshape(B, -1, n_kv, hd)       # [B, L, n_kv, hd]
    v = _values(s, "V", pages).reshape(B, -1, n_kv, hd)
    q, lim, b, slot = _padded(s)
    lim = torch.where(lim > 0, lim, torch.ones_like(lim))      # (rows that pad the batch)
    sc = torch.einsum("bsgjd,blgd->bgjsl", q, k) * (1.0 / math.sqrt(hd))
    dead = torch.arange(k.shape[1], device=b.device)[None, None, :] >= lim[:, :, None]      # [B, S, L]
    sc = sc.masked_fill_(dead[:, None, None], float("-inf"))
    sc = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    a = torch.einsum("bgjsl,blgd->bsgjd", sc, v) / sc.sum(-1).permute(0, 3, 1, 2)[..., None]
    s["out"][:s["rows"]] = a[b, slot].reshape(s["rows"], n_q, hd).to(s["out"].dtype)
    return s["out"]


def _new_slots(s):
    """[B, 1, slots]: the slot's key is one of the new rows'."""
    at = torch.arange(s["score"].shape[2], device=s["score"].device)[None, None, :]
    kl, n = s["kv_len"].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    return (at >= (kl - n)[:, None, None]) & (at < kl[:, None, None])


def _plain_weigh(s):
    n_kv, hd = s["K_pages"].shape[2:]
    B, n_q = s["table"].shape[0], s["Q"].shape[1]
    k = _values(s, "K", s["table"].long().clamp(min=0)).reshape(B, -1, n_kv, hd)
    q, lim, b, slot = _padded(s)
    lse = torch.zeros((B, s["max_new"], n_q), device=b.device)
    lse[b, slot] = s["lse"][:s["rows"]]
    lse = lse.view(B, -1, n_kv, n_q // n_kv).permute(0, 2, 3, 1)                              # [B, n_kv, G, S]
    w = torch.einsum("bsgjd,blgd->bgjsl", q, k) * (1.0 / math.sqrt(hd))
    w = w.sub_(lse[..., None]).exp_()
    dead = torch.arange(k.shape[1], device=b.device)[None, None, :] >= lim[:, :, None]
    w = w.masked_fill_(dead[:, None, None], 0.0).sum((2, 3))                                   # [B, n_kv, L]
    fresh = _new_slots(s)
    at = torch.arange(s["score"].shape[2], device=b.device)
    here = at < s["kv_len"].long()[:, None, None]
    s["score_out"].copy_(torch.where(here, torch.where(fresh, w, s["score"] + w), s["score_out"]))
    s["slot_pos"].copy_(torch.where(fresh, (at + s["pos_base"].long()[:, None])[:, None, :], s["slot_pos"].long()))
    return s["score_out"], s["slot_pos"]


def _move(s, which, src, dst, ok):
    """Rows src -> dst (slots [B, n_kv, M], where ok) of each key head; 8-bit rows take the scale of their new page."""
    pages = s[which + "_pages"]
    P, page, n_kv, _ = pages.shape
    b, g, i = ok.nonzero(as_tuple=True)
    ps, pd = (s["table"].long()[b, t[b, g, i] // page] for t in (src, dst))
    os_, od = src[b, g, i] % page, dst[b, g, i] % page
    if s[which + "_scale"] is None:
        pages[pd, od, g] = pages[ps, os_, g]
        return
    scale = s[which + "_scale"].view(torch.uint8)
    old, bits = scale.int(), pages.view(torch.uint8)
    rows = pages[ps, os_, g].float()
    into = torch.zeros((P, n_kv), dtype=torch.int32, device=b.device)          # the largest scale that comes in; 0: none
    into.view(-1).scatter_reduce_(0, pd * n_kv + g, old[ps, g] + 1, "amax")
    gone = torch.zeros((P, page, n_kv), dtype=torch.bool, device=b.device)
    gone[pd, od, g] = True
    # rows that stay in place: slots below the kept length that are not moved onto
    B, slots = s["table"].shape[0], s["score"].shape[2]
    at = torch.arange(slots, device=b.device)
    alive = at[None, :] < torch.minimum(s["keep"].long(), s["kv_len"].long())[:, None]
    owner = s["table"].long().clamp(min=0).repeat_interleave(page, 1)[:, :slots]
    live = torch.zeros((P, page), dtype=torch.bool, device=b.device)
    ab, aj = alive.nonzero(as_tuple=True)
    live[owner[ab, aj], aj % page] = True
    stay = live[:, :, None] & ~gone
    now = torch.where(stay.any(1), torch.maximum(old, into - 1), into - 1)
    now = torch.where(into > 0, now, old)
    grown = (now > old).any(1).nonzero()[:, 0]
    moved = pages[grown].float() * torch.exp2((old - now)[grown].float())[:, None, :, None]
    pick = (stay & (now > old)[:, None, :])[grown]
    bits[grown] = torch.where(pick[..., None], moved.to(pages.dtype).view(torch.uint8), bits[grown])
    bits[pd, od, g] = (rows * torch.exp2((old[ps, g] - now[pd, g]).float())[:, None]).to(pages.dtype).view(torch.uint8)
    scale.copy_(now)


def _plain_evict(s):
    sc, tag = s["score"], s["slot_pos"].long()
    B, n_kv, slots = sc.shape
    dev = sc.device
    at = torch.arange(slots, device=dev)[None, None, :]
    L, keep = s["kv_len"].long()[:, None, None], s["keep"].long()[:, None, None]
    here = at < L
    safe = here & (tag >= L + s["pos_base"].long()[:, None, None] - s["case"]["recent"])
    v = torch.where(here, sc, torch.full_like(sc, float("-inf")))
    order = torch.sort(v, dim=-1, descending=True, stable=True).indices
    kind = here.to(torch.int8) + safe.to(torch.int8)
    order = order.gather(-1, torch.sort(kind.gather(-1, order), dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, at.expand_as(order).contiguous())
    stays = here & (rank < keep)
    hole, source = (at < torch.minimum(keep, L)) & ~stays, (at >= keep) & stays
    n = hole.sum(-1)
    M = max(1, slots - s["case"]["keep"])
    # the slots of a mask in ascending order, [B, n_kv, M]
    src = torch.sort(torch.where(source, at, at + slots), -1).values[..., :M]
    dst = torch.sort(torch.where(hole, at, at + slots), -1).values[..., :M]
    ok = torch.arange(src.shape[-1], device=dev)[None, None, :] < n[..., None]
    src, dst = torch.where(ok, src, 0), torch.where(ok, dst, 0)
    _move(s, "K", src, dst, ok)
    _move(s, "V", src, dst, ok)
    so, to, lo, po = s["out"]
    left = at < torch.minimum(keep, L)
    b, g, i = ok.nonzero(as_tuple=True)
    new_s, new_t = sc.clone(), s["slot_pos"].clone()
    new_s[b, g, dst[b, g, i]] = sc[b, g, src[b, g, i]]
    new_t[b, g, dst[b, g, i]] = s["slot_pos"][b, g, src[b, g, i]]
    so.copy_(torch.where(left, new_s, so))
    to.copy_(torch.where(left, new_t, to))
    lo.copy_(torch.minimum(s["keep"], s["kv_len"]))
    po.copy_(s["pos_base"] + (s["kv_len"] - s["keep"]).clamp(min=0))
    return s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"], so, to, lo, po


def run(state):
    op = state["case"]["op"]
    s = state
    if own:
        from sparse_kv_cache_rank_gb300 import binding as B
        if op == "append":
            B.dllm_paged_append_f8(s["K"], s["V"], s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"], s["table"],
                                   s["q_start"], s["kv_len"], Q=s["Q"], Q_out=s["out"], gamma_q=s["gq"], gamma_k=s["gk"],
                                   eps=1e-6, inv_freq=s["inv_freq"])
            return s["out"], s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"]
        if op == "attend":
            return B.dllm_paged_attention_f8(s["Q"], s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"], s["table"],
                                             s["q_start"], s["kv_len"], s["max_new"], mask_block=s["case"]["mask"], A=s["out"])
        if op == "weigh":
            B.dllm_paged_weights(s["Q"], s["K_pages"], s["table"], s["q_start"], s["kv_len"], s["max_new"], s["lse"],
                                 s["score"], slot_pos=s["slot_pos"], K_scale=s["K_scale"], mask_block=s["case"]["mask"],
                                 pos_base=s["pos_base"], score_out=s["score_out"])
            return s["score_out"], s["slot_pos"]
        B.dllm_paged_evict(s["K_pages"], s["V_pages"], s["table"], s["kv_len"], s["keep"], s["score"], s["slot_pos"],
                           recent=s["case"]["recent"], pos_base=s["pos_base"], K_scale=s["K_scale"], V_scale=s["V_scale"],
                           out=s["out"])
        return s["K_pages"], s["V_pages"], s["K_scale"], s["V_scale"], *s["out"]
    return {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}[op](s)


# ---------------------------------------------------------------------------- 64 bits
def _dense(s, which, b, k):
    """Keys or values of sequence b, [k, n_kv, hd] in 64 bits."""
    pages = s[which + "_pages"]
    pg = s["table"][b, :-(-k // pages.shape[1])].long()
    x = pages[pg].double()
    if s[which + "_scale"] is not None:
        x = x * s[which + "_scale"].double()[pg][:, None, :, None]
    return x.reshape(-1, *pages.shape[2:])[:k]


def _exact_append(s, new, kv):
    page, hd = s["K_pages"].shape[1], s["K_pages"].shape[3]
    out = s["out"].double()
    res = {n: (s[n + "_pages"].double(), s[n + "_scale"].double()) for n in ("K", "V")}

    def turned(x, gamma, pos):
        x = x.double()
        if gamma is not None:
            x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-6) * gamma.double()
        ang = pos[:, None, None] * s["inv_freq"].double()
        z = torch.complex(x[..., :hd // 2], x[..., hd // 2:]) * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)

    at = 0
    for b, (n, k) in enumerate(zip(new, kv)):
        pos = torch.arange(k - n, k, device=out.device)
        out[at:at + n] = turned(s["Q"][at:at + n], s["gq"], pos.double())
        rows = {"K": turned(s["K"][at:at + n], s["gk"], pos.double()), "V": s["V"][at:at + n].double()}
        table = s["table"][b].tolist()
        for p in range((k - n) // page, (k - 1) // page + 1):
            lo, hi = max(k - n, p * page), min(k, (p + 1) * page)
            for name, x in rows.items():
                codes, scale = res[name]
                x = x[lo - (k - n):hi - (k - n)]
                e = torch.ceil(torch.log2(x.abs().amax((0, 2)) / MAX_CODE)).clamp(E_MIN, E_MAX)
                f = torch.exp2(e)
                if lo > p * page:
                    f = torch.maximum(f, scale[table[p]])
                    codes[table[p], :lo - p * page] *= (scale[table[p]] / f)[:, None]
                scale[table[p]] = f
                codes[table[p], lo - p * page:hi - p * page] = x / f[:, None]
        at += n
    return out, res["K"][0], res["V"][0], res["K"][1], res["V"][1]


def _exact_evict(s, case, kv):
    B, n_kv, slots = s["score"].shape
    page, f8 = case["page"], case["dtype"] == "f8"
    K, V = (None, None) if f8 else (s["K_pages"].double(), s["V_pages"].double())
    so, to, lo, po = (t.clone() for t in s["out"])
    score, tag, base = s["score"].cpu(), s["slot_pos"].cpu(), s["pos_base"].tolist()
    table = s["table"].long()
    so, to = so.cpu(), to.cpu()
    for b, k in enumerate(kv):
        keep = min(case["keep"], k)
        for g in range(n_kv):
            sc, tg = score[b, g, :k].tolist(), tag[b, g, :k].tolist()
            order = sorted(range(k), key=lambda j: (tg[j] < k + base[b] - case["recent"], -sc[j], j))
            stays = set(order[:keep])
            dst = [j for j in range(keep) if j not in stays]
            src = sorted(j for j in stays if j >= keep)
            slot = list(range(keep))
            for i, j in zip(dst, src):
                slot[i] = j
            so[b, g, :keep], to[b, g, :keep] = score[b, g][slot], tag[b, g][slot]
            if dst and not f8:
                d, j = torch.tensor(dst, device=table.device), torch.tensor(src, device=table.device)
                for x in (K, V):
                    x[table[b, d // page], d % page, g] = x[table[b, j // page], j % page, g]
        lo[b], po[b] = keep, base[b] + k - keep
    return K, V, None, None, so.double(), to, lo, po


def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence, page or head at a time."""
    s = prepare(case, seed)
    new, kv = _lengths(case)
    if case["op"] == "append":
        return _exact_append(s, new, kv)
    if case["op"] == "evict":
        return _exact_evict(s, case, kv)
    n_q, n_kv, hd, m = case["n_q"], case["n_kv"], case["hd"], case["mask"]
    weigh = case["op"] == "weigh"
    out = (s["score_out"] if weigh else s["out"]).double()
    at = 0
    for b, (n, k) in enumerate(zip(new, kv)):
        K = _dense(s, "K", b, k)
        V = None if weigh else _dense(s, "V", b, k)
        j, pos = torch.arange(k, device=out.device), torch.arange(k - n, k, device=out.device)
        seen = torch.ones((n, k), dtype=torch.bool, device=out.device) if m == 0 else j[None, :] // m <= pos[:, None] // m
        if weigh:
            out[b, :, :k] = torch.where(j < k - n, s["score"][b, :, :k].double(), 0.0)
            s["slot_pos"][b, :, k - n:k] = (pos + s["pos_base"][b]).to(torch.int32)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            sc = torch.where(seen, s["Q"][at:at + n, h].double() @ K[:, g].T / hd ** 0.5, float("-inf"))
            if weigh:
                out[b, g, :k] += torch.exp(sc - s["lse"][at:at + n, h].double()[:, None]).sum(0)
            else:
                out[at:at + n, h] = torch.softmax(sc, -1) @ V[:, g]
        at += n
    return (out, s["slot_pos"]) if weigh else out
