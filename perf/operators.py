"""What the paged-serving operators are measured on.

A decode step over a paged cache runs three of the library's operators: the new rows' queries
and keys are normalised, rotated and appended to the pages (dllm_paged_append), the queries
attend over the pages (dllm_paged_attention), and the vocabulary step draws a token per row
from given random numbers (dllm_sample).  Each case below is one pass through one of them.

Where `own` is false, `run` computes the operators in their plain form (elementary torch
operations); where it is true, it makes the library's calls on the same state.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- the cases
def _append(name, B, new, kv, ragged, n_q, n_kv, hd, page, src, dtype, norm, pad=0):
    return {"name": name, "op": "append", "B": B, "new": new, "kv": kv, "ragged": ragged, "n_q": n_q, "n_kv": n_kv,
            "hd": hd, "page": page, "src": src, "dtype": dtype, "norm": norm, "pad": pad}


def _attend(name, B, new, kv, ragged, n_q, n_kv, hd, page, dtype, mask, pad=0):
    return {"name": name, "op": "attend", "B": B, "new": new, "kv": kv, "ragged": ragged, "n_q": n_q, "n_kv": n_kv,
            "hd": hd, "page": page, "dtype": dtype, "mask": mask, "pad": pad}


def _sample(name, B, M, V, dtype, t, top_k, top_p, min_p, std, mixed):
    return {"name": name, "op": "sample", "B": B, "M": M, "V": V, "dtype": dtype, "t": t, "top_k": top_k,
            "top_p": top_p, "min_p": min_p, "std": std, "mixed": mixed}


def listed():
    return [
        # the current block of one LLaDA-8B-shaped sequence enters the cache (latency)
        _append("append_block", 1, 32, 1024, 0, 32, 32, 128, 64, "bf16", "bf16", False),
        # one new token each of 64 Dream-7B-shaped sequences, fp32 rows of the projection, normed heads
        _append("append_tokens", 64, 1, 2048, 50, 28, 4, 128, 16, "f32", "bf16", True),
        # four ragged prompts, the whole fused projection output, batch padded to a fixed row count
        _append("append_prompts", 4, 2048, 2048, 30, 32, 32, 128, 64, "bf16", "bf16", True, 96),
        # a block of masked tokens of one LLaDA-8B-shaped sequence over its cache (latency)
        _attend("attend_block", 1, 32, 1024, 0, 32, 32, 128, 64, "bf16", 0),
        # single tokens of 64 ragged sequences, grouped heads, small pages
        _attend("attend_tokens", 64, 1, 8192, 50, 28, 4, 128, 16, "bf16", 1, 3),
        # blocks of 16 ragged sequences, one query head per key head
        _attend("attend_blocks", 16, 32, 4096, 50, 32, 32, 128, 64, "bf16", 0),
        # the second half of two long prompts, blocks of 32 see the blocks up to their own
        _attend("attend_prompts", 2, 4096, 8192, 10, 28, 4, 128, 128, "bf16", 32),
        # the tiny fp32 layer's heads over an odd-sized cache
        _attend("attend_f32", 4, 32, 2001, 20, 8, 8, 64, 32, "f32", 1),
        # one row of a small vocabulary (latency)
        _sample("sample_row", 1, 1, 4096, "f32", 1.0, 0, 0.9, 0.0, 3.0, False),
        # the blocks of 8 LLaDA-8B-shaped sequences, all three filters
        _sample("sample_blocks", 8, 32, 126464, "f32", 0.8, 50, 0.95, 0.02, 3.0, False),
        # one row each of 64 requests with their own settings, a few of them greedy
        _sample("sample_requests", 64, 1, 152064, "bf16", 0.7, 0, 0.9, 0.0, 3.0, True),
        # the same vocabulary without a filter: every token can be drawn
        _sample("sample_open", 8, 32, 152064, "f32", 1.0, 0, 1.0, 0.0, 3.0, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    if op == "sample":
        V = _log(rng, 1000, 152064)
        rows = _log(rng, 1, min(256, 8 * 32 * 126464 // V))
        B = max(1, rows // rng.choice([1, 1, 8, 32]))
        M = max(1, rows // B)
        return _sample(None, B, M, V, rng.choice(["f32", "f32", "bf16"]), rng.choice([0.6, 0.8, 1.0, 1.2]),
                       rng.choice([0, 0, 1, 20, 50, _log(rng, 2, 4000)]), rng.choice([1.0, 0.8, 0.9, 0.95, 0.99]),
                       rng.choice([0.0, 0.0, 0.02, 0.1]), rng.choice([1.0, 2.0, 3.0]), rng.random() < 0.3)
    n_q, n_kv, hd = rng.choice([(32, 32, 128), (28, 4, 128), (8, 8, 64), (16, 2, 128), (12, 4, 64), (8, 1, 128)])
    page = rng.choice([16, 32, 64, 128])
    f32 = rng.random() < 0.2
    B = _log(rng, 1, 64)
    if op == "append":
        new = _log(rng, 1, max(1, 6000 // B))
        kv = new + rng.choice([0, _log(rng, 1, 8192)])
        src, dtype = ("f32", "f32") if f32 else (rng.choice(["bf16", "bf16", "f32"]), "bf16")
        return _append(None, B, new, kv, rng.choice([0, 20, 50]), n_q, n_kv, hd, page, src, dtype, rng.random() < 0.5,
                       rng.choice([0, 0, 7]))
    new = rng.choice([1, _log(rng, 2, 40), _log(rng, 8, 4096)])
    most = 2 * 4096 * 8192 * 28 * 128 // (B * new * n_q * hd)
    most = min(most, 64 * 8192 * 4 // (B * n_kv), 65536)
    if f32:
        most = min(most // 64, 4096)
        new = min(new, 64)
    kv = max(new, _log(rng, 16, max(17, most)))
    return _attend(None, B, new, kv, rng.choice([0, 20, 50]), n_q, n_kv, hd, page, "f32" if f32 else "bf16",
                   rng.choice([0, 1, 32]), rng.choice([0, 0, 5]))


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
    if case["op"] == "sample":
        n = case["B"] * case["M"] * case["V"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["B"] * (16 + 12 * case["M"]), "flops": 4 * n}
    new, kv = _lengths(case)
    hd, n_q, n_kv = case["hd"], case["n_q"], case["n_kv"]
    el = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        src = 2 if case["src"] == "bf16" else 4
        heads = n_q + 2 * n_kv
        return {"bytes": sum(new) * heads * hd * (src + el) + 4 * (sum(new) // case["page"] + 3 * case["B"] + hd),
                "flops": sum(new) * (n_q + n_kv) * hd * (7 if case["norm"] else 3)}
    return {"bytes": 2 * sum(new) * n_q * hd * el + 2 * sum(kv) * n_kv * hd * el + 4 * (sum(kv) // case["page"] + 3 * case["B"]),
            "flops": 4 * _visible(case, new, kv) * n_q * hd}


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=dev, dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "sample":
        B, M, V = case["B"], case["M"], case["V"]
        s["logits"] = (randn(B, M, V) * case["std"]).to(DT[case["dtype"]])
        s["u"] = torch.rand((B, M), generator=g, device=dev)

        def each(base, spread):   # one setting per sequence; `mixed`: each request brings its own
            v = torch.full((B,), float(base), device=dev)
            return v * (1 + spread * (2 * torch.rand((B,), generator=g, device=dev) - 1)) if case["mixed"] else v

        s["temperature"] = each(case["t"], 0.3)
        s["top_p"] = each(case["top_p"], 0.08)
        s["min_p"] = each(case["min_p"], 0.3)
        s["top_k"] = each(case["top_k"], 0.5).to(torch.int32)
        if case["mixed"]:
            s["temperature"][::8] = 0.0
        s["out"] = (torch.empty((B, M), dtype=torch.int32, device=dev), torch.empty((B, M), device=dev))
        return s
    new, kv = _lengths(case)
    hd, n_q, n_kv, page, B = case["hd"], case["n_q"], case["n_kv"], case["page"], case["B"]
    dt = DT[case["dtype"]]
    T = sum(new) + case["pad"]
    need = [-(-k // page) for k in kv]
    P = sum(need) + 2
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["table"] = table.to(dev)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32).to(dev)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32).to(dev)
    s["max_new"] = max(new)
    s["K_pages"] = randn(P, page, n_kv, hd).to(dt)
    s["V_pages"] = randn(P, page, n_kv, hd).to(dt)
    s["out"] = torch.zeros((T, n_q, hd), device=dev, dtype=dt)
    if case["op"] == "append":
        qkv = randn(T, n_q + 2 * n_kv, hd).to(DT[case["src"]])   # the fused projection's output
        s["Q"], s["K"], s["V"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        s["gq"] = s["gk"] = None
        if case["norm"]:
            s["gq"] = (1 + 0.1 * randn(hd)).to(dt)
            s["gk"] = (1 + 0.1 * randn(hd)).to(dt)
        s["inv_freq"] = (10000.0 ** (-2 * torch.arange(hd // 2, dtype=torch.float64) / hd)).float().to(dev)
        # host sizes of the plain form's index arithmetic
        s["rows"] = sum(new)
    else:
        s["Q"] = (randn(T, n_q, hd) * 1.5).to(dt)
        s["rows"] = sum(new)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _where(s):
    """Sequence and position of every new row."""
    t = torch.arange(s["rows"], device=s["q_start"].device)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    pos = t - s["q_start"].long()[b] + s["kv_len"].long()[b] - (s["q_start"].long()[b + 1] - s["q_start"].long()[b])
    return b, pos


def _normed(x, gamma, eps):
    if gamma is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.float()


def _rotated(x, cos, sin):
    h = x.shape[-1] // 2
    a, c = x[..., :h], x[..., h:]
    return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)


def _plain_append(s):
    b, pos = _where(s)
    ang = pos.double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    n = s["rows"]
    q = _rotated(_normed(s["Q"][:n].float(), s["gq"], 1e-6), cos, sin)
    k = _rotated(_normed(s["K"][:n].float(), s["gk"], 1e-6), cos, sin)
    page = s["K_pages"].shape[1]
    at = s["table"].long()[b, pos // page], pos % page
    s["K_pages"][at] = k.to(s["K_pages"].dtype)
    s["V_pages"][at] = s["V"][:n].to(s["V_pages"].dtype)
    s["out"][:n] = q.to(s["out"].dtype)
    return s["out"], s["K_pages"], s["V_pages"]


def _plain_attend(s):
    n_kv, hd, page = s["K_pages"].shape[2], s["K_pages"].shape[3], s["K_pages"].shape[1]
    B, n_q = s["table"].shape[0], s["Q"].shape[1]
    pages = s["table"].long().clamp(min=0)
    k = s["K_pages"][pages].float().reshape(B, -1, n_kv, hd)       # [B, L, n_kv, hd]
    v = s["V_pages"][pages].float().reshape(B, -1, n_kv, hd)
    b, pos = _where(s)
    slot = torch.arange(s["rows"], device=b.device) - s["q_start"].long()[b]
    q = torch.zeros((B, s["max_new"], n_q, hd), device=b.device)
    q[b, slot] = s["Q"][:s["rows"]].float()
    q = q.view(B, s["max_new"], n_kv, n_q // n_kv, hd)
    m = s["case"]["mask"]
    lim = s["kv_len"].long()[:, None].expand(B, s["max_new"]).clone()
    if m > 0:
        lim[b, slot] = torch.minimum(s["kv_len"].long()[b], (pos // m + 1) * m)
    sc = torch.einsum("bsgjd,blgd->bgjsl", q, k) * (1.0 / math.sqrt(hd))
    dead = torch.arange(k.shape[1], device=b.device)[None, None, :] >= lim[:, :, None]      # [B, S, L]
    sc = sc.masked_fill_(dead[:, None, None], float("-inf"))
    sc = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    a = torch.einsum("bgjsl,blgd->bsgjd", sc, v) / sc.sum(-1).permute(0, 3, 1, 2)[..., None]
    s["out"][:s["rows"]] = a[b, slot].reshape(s["rows"], n_q, hd).to(s["out"].dtype)
    return s["out"]


def _plain_sample(s):
    B, M, V = s["logits"].shape
    t = s["temperature"]
    greedy = (t <= 0)[:, None]
    inv = torch.where(t > 0, 1.0 / t, torch.ones_like(t))
    z = s["logits"].float() * inv[:, None, None]                    # scaled logits, fp32
    top = z.amax(-1, keepdim=True)
    first = (z == top).to(torch.int8).argmax(-1)                    # lowest index of the maximum
    zs, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = (zs.double() - top.double()).exp()
    rank = torch.arange(V, device=z.device)
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), torch.full_like(s["top_k"].long(), V))[:, None, None]
    w = torch.where(rank < k, w, torch.zeros((), dtype=torch.float64, device=z.device))
    cum = w.cumsum(-1)
    keep = (cum - w < s["top_p"].double()[:, None, None] * cum[..., -1:]) | (s["top_p"] >= 1)[:, None, None]
    keep &= (w >= s["min_p"].double()[:, None, None]) & (w > 0)
    keep[..., 0] = True
    kept = torch.zeros((B, M, V), dtype=torch.float64, device=z.device)
    kept.scatter_(-1, order, torch.where(keep, w, torch.zeros_like(w)))
    run_ = kept.cumsum(-1)
    total = run_[..., -1]
    tok = (run_ <= (s["u"].double() * total)[..., None]).sum(-1).clamp(max=V - 1)
    prob = kept.gather(-1, tok[..., None])[..., 0] / total
    s["out"][0].copy_(torch.where(greedy, first, tok))
    s["out"][1].copy_(torch.where(greedy, torch.ones_like(prob), prob))
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        from sparse_kv_cache_rank_gb300 import binding as B
        s = state
        if op == "append":
            B.dllm_paged_append(s["K"], s["V"], s["K_pages"], s["V_pages"], s["table"], s["q_start"], s["kv_len"],
                                Q=s["Q"], Q_out=s["out"], gamma_q=s["gq"], gamma_k=s["gk"], eps=1e-6,
                                inv_freq=s["inv_freq"])
            return s["out"], s["K_pages"], s["V_pages"]
        if op == "attend":
            return B.dllm_paged_attention(s["Q"], s["K_pages"], s["V_pages"], s["table"], s["q_start"], s["kv_len"],
                                          s["max_new"], mask_block=s["case"]["mask"], A=s["out"])
        return B.dllm_sample(s["logits"], s["u"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"], out=s["out"])
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state) if op == "attend" else _plain_sample(state)


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence or row at a time."""
    s = prepare(case, seed)
    if case["op"] == "sample":
        B, M, V = s["logits"].shape
        tok, prob = torch.zeros((B, M), dtype=torch.int32), torch.zeros((B, M), dtype=torch.float64)
        for b in range(B):
            t, k, p, mp = (float(s[n][b]) for n in ("temperature", "top_k", "top_p", "min_p"))
            for i in range(M):
                l = s["logits"][b, i].float()
                if t <= 0:
                    tok[b, i], prob[b, i] = int((l == l.max()).nonzero()[0]), 1.0
                    continue
                z = (l * (1.0 / s["temperature"][b])).double()      # the definition's fp32 scaled logit
                w = torch.exp(z - z.max())
                # descending weight, ties by index: a stable sort of the negated values
                idx = torch.sort(-z, stable=True).indices
                ws = w[idx]
                if 0 < k < V:
                    ws = ws[:int(k)]
                cum = torch.cumsum(ws, 0)
                n = len(ws)
                if p < 1:
                    n = min(n, int((cum - ws < p * cum[-1]).sum()))
                if mp > 0:
                    n = min(n, int((ws >= mp).sum()))
                ids = torch.sort(idx[:max(n, 1)]).values
                c = torch.cumsum(w[ids], 0)
                j = int(torch.searchsorted(c, float(s["u"][b, i]) * c[-1], right=True).clamp(max=len(ids) - 1))
                tok[b, i], prob[b, i] = int(ids[j]), float(w[ids[j]] / c[-1])
        return tok, prob
    new, kv = _lengths(case)
    page, hd, n_q, n_kv = case["page"], case["hd"], case["n_q"], case["n_kv"]
    if case["op"] == "append":
        out, kp, vp = (s[n].double() for n in ("out", "K_pages", "V_pages"))

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
            pg = s["table"][b].long()[pos // page]
            kp[pg, pos % page] = turned(s["K"][at:at + n], s["gk"], pos.double())
            vp[pg, pos % page] = s["V"][at:at + n].double()
            at += n
        return out, kp, vp
    out, m = s["out"].double(), case["mask"]
    at = 0
    for b, (n, k) in enumerate(zip(new, kv)):
        pg = s["table"][b, :-(-k // page)].long()
        K = s["K_pages"][pg].reshape(-1, n_kv, hd)[:k].double()
        V = s["V_pages"][pg].reshape(-1, n_kv, hd)[:k].double()
        pos = torch.arange(k - n, k, device=out.device)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            sc = s["Q"][at:at + n, h].double() @ K[:, g].T / hd ** 0.5
            if m > 0:
                j = torch.arange(k, device=out.device)
                sc = torch.where(j[None, :] // m <= pos[:, None] // m, sc, float("-inf"))
            out[at:at + n, h] = torch.softmax(sc, -1) @ V[:, g]
        at += n
    return out
