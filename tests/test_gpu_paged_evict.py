"""GPU parity of the keys' accumulated attention weights and of the eviction by them with their fp64 definitions, over
bf16, fp32 and 8-bit pages; and a serving loop that appends, attends, weighs and evicts.

Tolerances: a weight exp(s - lse) in fp32 carries hd 2^-23 |q| |k| scale of its score, 2^-22 (|s| + |lse|) for their
products with log2 e, 1e-5 for nothing else than the exponential's 2^-22 and n additions of 2^-24 each.  Moved rows,
positions and lengths are exact; 8-bit codes that are rounded anew are compared with the definition's rounding.
"""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_gpu_paged import BF, F32, B, Batch, dev, host  # noqa: F401  (B: the library fixture)
from test_gpu_paged_f8 import E4M3, E8M0, Batch8, exps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F8 = "f8"
KINDS = [BF, F32, F8]
IDS = ["bf16", "f32", "f8"]


def make(seed, seqs, n_q, n_kv, hd, page, kind, **kw):
    S = Batch8(seed, seqs, n_q, n_kv, hd, page, spread=2, **kw) if kind == F8 else Batch(seed, seqs, n_q, n_kv, hd, page, kind, **kw)
    S.kind = kind
    S.qdt = BF if kind == F8 else kind
    S.Ks, S.Vs = (S.Ks, S.Vs) if kind == F8 else (None, None)
    return S


def keys_of(S):
    return S.values()[0] if S.kind == F8 else host(S.Kp)


# ---------------------------------------------------------------------------- weights
WEIGH = [
    # seqs (new, keys), n_q, n_kv, hd, page, mask_block, pad
    ([(1, 1)], 1, 1, 64, 8, 0, 0),
    ([(32, 1024)], 4, 4, 128, 64, 0, 0),
    ([(1, 77), (1, 16), (0, 40), (1, 3000), (1, 1), (1, 129)], 28, 4, 128, 16, 1, 3),
    ([(67, 130), (0, 0), (5, 5), (33, 2100)], 6, 2, 64, 32, 1, 4),
    ([(300, 700), (129, 129), (1, 300)], 7, 1, 128, 128, 32, 0),
    ([(5, 3), (4, 0), (2, 2), (3, 200)], 4, 2, 128, 16, 1, 2),       # rows before position 0
    ([(40, 640)], 128, 1, 64, 64, 7, 0),                             # 128 heads share a key head
    ([(20, 500), (3, 256)], 2, 2, 64, 256, 1, 1),
    ([(2, 900), (4, 900)], 12, 3, 128, 8, 0, 0),
]


def weigh_case(B, i, kind, in_place=False):  # noqa: F811
    seqs, n_q, n_kv, hd, page, mb, pad = WEIGH[i]
    S = make(500 + i, seqs, n_q, n_kv, hd, page, kind, pad=pad)
    S.poison()
    q = S.g.standard_normal((S.T, n_q, hd), dtype=np.float32) * 1.5
    S.Q = dev(q, S.qdt)
    most = max(n for n, _ in seqs)
    lse = torch.full((S.T, n_q), 5.0, device="cuda")
    if kind == F8:
        B.dllm_paged_attention_f8(S.Q, S.Kp, S.Vp, S.Ks, S.Vs, *S.d, most, mask_block=mb, lse=lse)
    else:
        B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, most, mask_block=mb, lse=lse)
    slots = S.table.shape[1] * page + 5
    score = torch.from_numpy(S.g.random((len(seqs), n_kv, slots)).astype(np.float32)).cuda()
    tags = torch.full((len(seqs), n_kv, slots), -7, dtype=torch.int32, device="cuda")
    base = torch.from_numpy(S.g.integers(0, 900, len(seqs)).astype(np.int32)).cuda()
    before, out = score.clone(), score if in_place else torch.full_like(score, 3.0)
    got = B.dllm_paged_weights(S.Q, S.Kp, *S.d, most, lse, score, slot_pos=tags, K_scale=S.Ks, mask_block=mb, pos_base=base,
                               score_out=None if in_place else out)
    assert got is out and B.check_status() == 0
    K = np.nan_to_num(keys_of(S), nan=0.0)
    ref, tag, mag = paged.weights(host(S.Q), K, S.table, S.q_start, S.kv_len, host(lse), host(before),
                                  tags.clone().fill_(-7).cpu().numpy(), mb, None, base.cpu().numpy())
    assert np.array_equal(tags.cpu().numpy(), tag)
    for b, (n, k) in enumerate(seqs):
        L = min(k, slots) if n else 0
        assert torch.equal(out[b, :, L:], before[b, :, L:] if in_place else torch.full_like(out[b, :, L:], 3.0))
        kn = np.linalg.norm(K[S.used()], axis=-1).max() if S_used_any(S) else 0.0
        ds = hd * 2.0 ** -23 * (np.linalg.norm(host(S.Q), axis=-1).max() if S.T else 0.0) * kn * hd ** -0.5
        tol = mag[b, :, :L] * (ds + 2.0 ** -21 + n * n_q * 2.0 ** -24) + 2.0 ** -23 * np.abs(ref[b, :, :L]) + 1e-30
        err = np.abs(host(out)[b, :, :L] - ref[b, :, :L])
        assert (err <= tol).all(), (b, (err - tol).max())
    return S, lse, score, out, most, mb


def S_used_any(S):
    if not hasattr(S, "used"):
        used = np.zeros((S.P, S.page), bool)
        for b, (_, k) in enumerate(S.seqs):
            for j in range(min(k, S.table.shape[1] * S.page)):
                p = S.table[b, j // S.page]
                if 0 <= p < S.P:
                    used[p, j % S.page] = True
        S.used = lambda: used
    return S.used().any()


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("i", range(len(WEIGH)))
def test_weights_parity(B, i, kind):  # noqa: F811
    S, lse, score, out, most, mb = weigh_case(B, i, kind, in_place=i % 2 == 1)
    if i % 2 == 0:                       # the same sums every time
        again = torch.full_like(out, 3.0)
        B.dllm_paged_weights(S.Q, S.Kp, *S.d, most, lse, score, K_scale=S.Ks, mask_block=mb, score_out=again)
        assert torch.equal(again, out)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_weights_of_all_rows_sum_to_their_number(B, kind):  # noqa: F811
    """Each row and head spreads a weight of 1 over the keys that it sees."""
    seqs = [(3, 1000), (70, 400), (1, 9)]
    S = make(540, seqs, 8, 2, 64, 16, kind)
    S.Q = dev(S.g.standard_normal((S.T, 8, 64), dtype=np.float32), S.qdt)
    lse, slots = torch.empty((S.T, 8), device="cuda"), 1008
    call = B.dllm_paged_attention_f8 if kind == F8 else B.dllm_paged_attention
    args = (S.Kp, S.Vp, S.Ks, S.Vs) if kind == F8 else (S.Kp, S.Vp)
    call(S.Q, *args, *S.d, 70, mask_block=1, lse=lse)
    score = torch.zeros((3, 2, slots), device="cuda")
    B.dllm_paged_weights(S.Q, S.Kp, *S.d, 70, lse, score, K_scale=S.Ks, mask_block=1)
    total = host(score).sum(-1)
    want = np.array([n for n, _ in seqs])[:, None] * 4.0
    # 8 bits: the attention's lse has its queries in two parts (2^-17 of the largest element), here they are whole
    assert np.abs(total - want).max() <= want.max() * (1e-4 if kind == F8 else 1e-5)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_weights_rows_that_are_no_numbers_absent_pages_and_short_arrays(B, kind):  # noqa: F811
    seqs = [(3, 300), (2, 90)]
    S = make(541, seqs, 4, 2, 64, 16, kind)
    q = S.g.standard_normal((S.T, 4, 64)).astype(np.float32)
    S.Q = dev(q, S.qdt)
    S.Q[1, 2, 5] = float("nan")
    S.Q[3, 0, 0] = float("inf")
    table = S.table.copy()
    table[0, 3], table[1, 0] = -1, S.P
    d = [torch.from_numpy(table).cuda(), *S.d[1:]]
    lse = torch.from_numpy(S.g.random((S.T, 4)).astype(np.float32) + 6).cuda()
    lse[1, 2], lse[3, 0], lse[0, 1] = float("nan"), float("nan"), -float("inf")
    slots = 250                                            # shorter than the first sequence
    score = torch.from_numpy(S.g.random((2, 2, slots)).astype(np.float32)).cuda()
    before = host(score)
    B.dllm_paged_weights(S.Q, S.Kp, *d, 3, lse, score, K_scale=S.Ks, mask_block=1)
    Q = np.nan_to_num(host(S.Q), nan=0.0, posinf=0.0)
    ref, _, mag = paged.weights(Q, keys_of(S), table, S.q_start, S.kv_len, host(lse), before, np.zeros(before.shape), 1)
    assert np.isfinite(host(score)).all()
    assert (np.abs(host(score) - ref) <= mag * 1e-4 + 1e-6).all() and B.check_status() == 0


# ---------------------------------------------------------------------------- eviction
EVICT = [
    # seqs (keys, keep), n_kv, hd, page, recent, spare slots
    ([(1, 1)], 1, 64, 8, 0, 0),
    ([(1, 0)], 1, 64, 8, 3, 0),
    ([(1056, 1024)], 4, 128, 64, 32, 0),
    ([(700, 350), (130, 200), (0, 5), (9000, 4500), (33, 1)], 2, 64, 16, 20, 7),
    ([(300, 299), (300, 150), (256, 255)], 3, 128, 128, 0, 0),
    ([(500, 100), (4097, 4096)], 1, 128, 256, 300, 1),          # more protected than may stay
    ([(5000, 17), (90, 45)], 8, 64, 32, 64, 0),
]


def state(S, kind, recent, slots, ties):
    """Scores (many alike where `ties`), positions in some order, bases."""
    Bn, n_kv = len(S.seqs), S.Kp.shape[2]
    sc = S.g.random((Bn, n_kv, slots)).astype(np.float32)
    if ties:
        sc = np.floor(sc * 5) - 2
        sc[sc == 0] = np.where(S.g.random((sc == 0).sum()) < 0.5, -0.0, 0.0)
        sc[S.g.random(sc.shape) < 0.1] = np.nan
        sc[S.g.random(sc.shape) < 0.02] = np.inf
        sc[S.g.random(sc.shape) < 0.02] = -np.inf
    base = S.g.integers(0, 1000, Bn).astype(np.int32)
    tag = np.zeros(sc.shape, np.int32)
    for b, (_, k) in enumerate(S.seqs):
        for g in range(n_kv):
            tag[b, g, :k] = S.g.permutation(k)[:slots] + base[b] if ties else np.arange(k)[:slots] + base[b]
    return sc, tag, base


def check_evicted(S, kind, got, before, plan, out, sc, tag, base, kv, keep):
    (k0, v0), (so, to, lo, po) = before, out
    page = S.page
    want = {"K": k0.copy(), "V": v0.copy()}
    e0 = {"K": S.Ke.copy(), "V": S.Ve.copy()} if kind == F8 else None
    e1 = {n: e.copy() for n, e in e0.items()} if kind == F8 else None
    so_w, to_w = sc.copy(), tag.copy()
    for (b, g), (K, moves) in plan.items():
        at = lambda j: (S.table[b, j // page], j % page)      # noqa: E731
        holes = {d for d, _ in moves}
        for n in ("K", "V"):
            if kind == F8:
                for pg in sorted({d // page for d, _ in moves}):
                    ins = [(d, s) for d, s in moves if d // page == pg]
                    rest = [j for j in range(pg * page, min((pg + 1) * page, K)) if j not in holes]
                    p = S.table[b, pg]
                    now = max([e0[n][at(s)[0], g] for _, s in ins] + ([e0[n][p, g]] if rest else []))
                    for j in rest:
                        want[n][p, j % page, g] = paged.e4m3(k0[p, j % page, g] * 2.0 ** (e0[n][p, g] - now)) if n == "K" else \
                            paged.e4m3(v0[p, j % page, g] * 2.0 ** (e0[n][p, g] - now))
                    for d, s in ins:
                        src = (k0 if n == "K" else v0)[at(s)[0], at(s)[1], g]
                        want[n][p, d % page, g] = paged.e4m3(src * 2.0 ** (e0[n][at(s)[0], g] - now))
                    e1[n][p, g] = now
            else:
                for d, s in moves:
                    want[n][at(d)[0], at(d)[1], g] = (k0 if n == "K" else v0)[at(s)[0], at(s)[1], g]
        for d, s in moves:
            so_w[b, g, d], to_w[b, g, d] = sc[b, g, s], tag[b, g, s]
        assert np.array_equal(so.cpu().numpy()[b, g, :K], so_w[b, g, :K], equal_nan=True)
        assert np.array_equal(to.cpu().numpy()[b, g, :K], to_w[b, g, :K])
    assert np.array_equal(host(got[0]), want["K"]) and np.array_equal(host(got[1]), want["V"])
    if kind == F8:
        assert np.array_equal(exps(S.Ks), e1["K"]) and np.array_equal(exps(S.Vs), e1["V"])
    L = np.minimum(kv, so.shape[2])
    K = np.minimum(np.maximum(keep, 0), L)
    assert np.array_equal(lo.cpu().numpy(), np.where(K < L, K, kv)) and np.array_equal(po.cpu().numpy(), base + L - K)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("ties", [False, True], ids=["apart", "ties"])
@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict_parity(B, i, ties, kind):  # noqa: F811
    seqs, n_kv, hd, page, recent, spare = EVICT[i]
    S = make(600 + i, [(0, k) for k, _ in seqs], n_kv, n_kv, hd, page, kind)
    slots = max(1, S.table.shape[1] * page + spare)
    sc, tag, base = state(S, kind, recent, slots, ties)
    keep = np.array([k for _, k in seqs], np.int32)
    plan = paged.evict(S.kv_len, keep, sc, tag, recent, base, S.table.shape[1] * page)
    t = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, base, keep)]
    before = (host(S.Kp), host(S.Vp))
    in_place = i % 2 == 0
    out = None if in_place else (torch.full_like(t[0], 9.0), torch.full_like(t[1], 9), torch.full_like(t[2], 9), torch.full_like(t[3], 9))
    got = B.dllm_paged_evict(S.Kp, S.Vp, S.d[0], t[2], t[4], t[0], t[1], recent=recent, pos_base=t[3], K_scale=S.Ks, V_scale=S.Vs, out=out)
    assert B.check_status() == 0
    check_evicted(S, kind, (S.Kp, S.Vp), before, plan, got, sc, tag, base, S.kv_len, keep)
    if not in_place:
        assert all((got[0][b, :, min(int(k), slots):] == 9).all() for b, k in enumerate(np.minimum(keep, S.kv_len)))


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_evict_without_bases_rows_without_pages_and_replay(B, kind):  # noqa: F811
    """A slot to fill or to move that lacks a page raises the status, the others move; a captured call follows new
    lengths and keeps."""
    S = make(620, [(0, 90), (0, 64)], 2, 2, 64, 16, kind)
    sc = S.g.random((2, 2, 96)).astype(np.float32)
    tag = np.tile(np.arange(96, dtype=np.int32), (2, 2, 1))
    sc[0, :, :16] -= 5.0                                  # page 0 of sequence 0: all holes
    keep = np.array([60, 64], np.int32)
    table = S.table.copy()
    table[0, 0] = -1
    plan = paged.evict(S.kv_len, keep, sc, tag, 0, None, 96)
    k0 = host(S.Kp)
    t = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, keep, table)]
    out = tuple(x.clone() for x in (t[0], t[1], t[2])) + (None,)
    B.dllm_paged_evict(S.Kp, S.Vp, t[4], t[2], t[3], t[0], t[1], K_scale=S.Ks, V_scale=S.Vs, out=out)
    assert B.check_status(reset=True) == B.STATUS_PAGE
    for (b, g), (K, moves) in plan.items():
        for d, s in moves:
            assert out[0][b, g, d] == sc[b, g, s]
            if table[b, d // 16] >= 0 and kind != F8:
                assert np.array_equal(host(S.Kp)[table[b, d // 16], d % 16, g], k0[table[b, s // 16], s % 16, g])
    assert np.array_equal(host(S.Kp)[S.table[0, 0]], k0[S.table[0, 0]])
    # capture
    S = make(621, [(0, 90), (0, 64)], 2, 2, 64, 16, kind)
    ins = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, keep)]
    out = tuple(torch.zeros_like(x) for x in ins[:3]) + (None,)
    k0, v0 = S.Kp.clone(), S.Vp.clone()
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        B.dllm_paged_evict(S.Kp, S.Vp, S.d[0], ins[2], ins[3], ins[0], ins[1], recent=4, K_scale=S.Ks, V_scale=S.Vs, out=out)
    for kv, kp in (([90, 64], [60, 64]), ([80, 50], [79, 3])):
        S.Kp.copy_(k0)
        S.Vp.copy_(v0)
        if kind == F8:
            S.upload()                                    # (scales)
            S.Kp, S.Vp, S.Ks, S.Vs = S.Kp, S.Vp, S.Ks, S.Vs
        ins[2].copy_(torch.tensor(kv, dtype=torch.int32))
        ins[3].copy_(torch.tensor(kp, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        plan = paged.evict(kv, kp, sc, tag, 4, None, 96)
        for (b, h), (K, moves) in plan.items():
            w = sc[b, h].copy()
            for d, s in moves:
                w[d] = sc[b, h, s]
            assert np.array_equal(out[0].cpu().numpy()[b, h, :K], w[:K])
        assert out[2].tolist() == [min(a, c) for a, c in zip(kv, kp)]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_append_attend_weigh_evict_as_a_server_runs_them(B, kind):  # noqa: F811
    """Two sequences grow by a prompt, blocks and tokens; each step appends at its true positions, attends, weighs, and
    gives up keys when there are more than a budget.  Every step is checked against the definitions on the device's own
    inputs of that step, and the first tokens' positions show that heads keep what they attend to."""
    n_q, n_kv, hd, page, budget, recent = 4, 2, 64, 16, 96, 24
    S = make(630, [(0, 160), (0, 160)], n_q, n_kv, hd, page, kind)
    g = S.g
    f = (10000.0 ** (-2 * np.arange(hd // 2) / hd)).astype(np.float32)
    ft = torch.from_numpy(f).cuda()
    slots = S.table.shape[1] * page
    score = torch.zeros((2, n_kv, slots), device="cuda")
    tags = torch.zeros((2, n_kv, slots), dtype=torch.int32, device="cuda")
    kv = torch.zeros(2, dtype=torch.int32, device="cuda")
    base = torch.zeros(2, dtype=torch.int32, device="cuda")
    keep = torch.full((2,), budget, dtype=torch.int32, device="cuda")
    seen = [0, 0]
    for step, new in enumerate(([37, 90], [32, 32], [32, 32], [1, 1], [1, 1])):
        qs_h = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        qs, T, most = torch.from_numpy(qs_h).cuda(), int(sum(new)), max(new)
        kv += torch.tensor(new, dtype=torch.int32, device="cuda")
        seen = [a + n for a, n in zip(seen, new)]
        assert (kv + base).tolist() == seen
        qkv = dev(g.standard_normal((T, n_q + 2 * n_kv, hd), dtype=np.float32), S.qdt)
        Q, K, V = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        table, cache = S.d[0], (S.Kp, S.Vp)
        if kind == F8:
            q = B.dllm_paged_append_f8(K, V, *cache, S.Ks, S.Vs, table, qs, kv, Q=Q, inv_freq=ft, pos_base=base)
        else:
            q = B.dllm_paged_append(K, V, *cache, table, qs, kv, Q=Q, inv_freq=ft, pos_base=base)
        rows = paged.rows_of(qs_h, kv.cpu().numpy(), T)
        want = np.stack([paged.rotated(host(Q)[t], p + base.tolist()[b], f) for t, (b, p) in enumerate(rows)])
        assert np.abs(host(q) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-5
        lse = torch.empty((T, n_q), device="cuda")
        if kind == F8:
            A = B.dllm_paged_attention_f8(q, *cache, S.Ks, S.Vs, table, qs, kv, most, mask_block=1, lse=lse)
            kvals, vvals = (host(c) * 2.0 ** exps(s)[:, None, :, None] for c, s in ((S.Kp, S.Ks), (S.Vp, S.Vs)))
        else:
            A = B.dllm_paged_attention(q, *cache, table, qs, kv, most, mask_block=1, lse=lse)
            kvals, vvals = host(S.Kp), host(S.Vp)
        Ar = paged.attention(host(q), kvals, vvals, S.table, qs_h, kv.cpu().numpy(), 1)[0]
        assert np.abs(host(A) - Ar).max() <= 0.02 * np.abs(Ar).max() + (1e-5 if kind == F32 else 0.01)
        before, tb = host(score), tags.cpu().numpy()
        B.dllm_paged_weights(q, S.Kp, table, qs, kv, most, lse, score, slot_pos=tags, K_scale=S.Ks, mask_block=1, pos_base=base)
        ref, tag, mag = paged.weights(host(q), kvals, S.table, qs_h, kv.cpu().numpy(), host(lse), before, tb, 1, None, base.cpu().numpy())
        assert (np.abs(host(score) - ref) <= 1e-4 * mag + 1e-6).all() and np.array_equal(tags.cpu().numpy(), tag)
        plan = paged.evict(kv.cpu().numpy(), keep.cpu().numpy(), score.cpu().numpy(), tag, recent, base.cpu().numpy(), slots)
        k0, sc0, kv0 = host(S.Kp), score.cpu().numpy(), kv.tolist()
        B.dllm_paged_evict(*cache, table, kv, keep, score, tags, recent=recent, pos_base=base, K_scale=S.Ks, V_scale=S.Vs)
        for (b, h), (n, moves) in plan.items():
            assert kv.tolist()[b] == n and base.tolist()[b] == seen[b] - n
            for d, s in moves:
                assert score[b, h, d] == sc0[b, h, s] and tags[b, h, d] == tag[b, h, s]
                if kind != F8:
                    assert np.array_equal(host(S.Kp)[S.table[b, d // page], d % page, h], k0[S.table[b, s // page], s % page, h])
            left = tags[b, h, :n].tolist()
            assert len(set(left)) == n and set(range(max(0, seen[b] - recent), seen[b])) <= set(left)
    assert B.check_status() == 0 and kv.tolist() == [budget] * 2


def test_writes_stay_inside_their_arrays(B):  # noqa: F811
    from test_gpu_guards import Guarded
    for kind in KINDS:
        seqs = [(3, 100), (1, 2000), (130, 130)]
        S = make(650, seqs, 6, 2, 128, 16, kind)
        G = Guarded(651)
        if kind == F8:
            u8 = [G.new(t.shape, torch.uint8, t.view(torch.uint8)) for t in (S.Kp, S.Vp, S.Ks, S.Vs)]
            Kp, Vp, Ks, Vs = u8[0].view(E4M3), u8[1].view(E4M3), u8[2].view(E8M0), u8[3].view(E8M0)
        else:
            Kp, Vp, Ks, Vs = G.new(S.Kp.shape, kind, S.Kp), G.new(S.Vp.shape, kind, S.Vp), None, None
        d = [G.new(t.shape, torch.int32, t) for t in S.d]
        Q = G.new((S.T, 6, 128), S.qdt, torch.randn((S.T, 6, 128)).to(S.qdt))
        lse = G.new((S.T, 6), F32, torch.full((S.T, 6), 6.0))
        slots = 2000
        sc, so = (G.new((3, 2, slots), F32, torch.rand((3, 2, slots))) for _ in range(2))
        tg = G.new((3, 2, slots), torch.int32, torch.zeros((3, 2, slots), dtype=torch.int32))
        base, keep = (G.new((3,), torch.int32, torch.tensor(x, dtype=torch.int32)) for x in ([5, 0, 7], [50, 1001, 0]))
        for most in (1, 3, 130):
            B.dllm_paged_weights(Q, Kp, *d, most, lse, sc, slot_pos=tg, K_scale=Ks, mask_block=1, pos_base=base, score_out=so)
        ws = G.new((B.dllm_paged_evict_workspace_bytes(3, 2, slots, Kp.dtype),), torch.uint8)
        B.dllm_paged_evict(Kp, Vp, d[0], d[2], keep, so, tg, recent=9, pos_base=base, K_scale=Ks, V_scale=Vs, ws=ws)
        assert B.check_status() == 0
        G.check()
