"""GPU parity of the eviction, compared whole (keys, values, scales, scores, positions, lengths), where
test_gpu_paged_evict.py and test_gpu_paged_smaller.py look at a part: replays of a captured call with new lengths, slots
whose rows should move but lack a page, selections past shared memory over 8-bit pages."""
import numpy as np
import pytest

from oracle import paged
from test_gpu_paged import B, host  # noqa: F401  (B: the library fixture)
from test_gpu_paged_evict import F8, IDS, KINDS, check_evicted, make, state
from test_gpu_paged_f8 import exps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_captured_eviction_follows_new_lengths(B, kind):  # noqa: F811
    S = make(720, [(0, 300), (0, 64), (0, 700)], 2, 2, 64, 16, kind)
    slots = S.table.shape[1] * 16
    sc, tag, base = state(S, kind, 4, slots, True)
    cache = [S.Kp, S.Vp] + ([S.Ks, S.Vs] if kind == F8 else [])
    kept = [t.view(torch.uint8).clone() for t in cache]
    t = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, base, S.kv_len)]
    out = tuple(torch.zeros_like(x) for x in t[:4])
    before = (host(S.Kp), host(S.Vp))
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        B.dllm_paged_evict(S.Kp, S.Vp, S.d[0], t[2], t[4], t[0], t[1], recent=4, pos_base=t[3], K_scale=S.Ks, V_scale=S.Vs, out=out)
    for kv, keep in (([300, 64, 700], [200, 64, 350]), ([80, 50, 0], [79, 3, 9]), ([299, 1, 513], [0, 0, 512]), ([5, 64, 700], [1, 33, 699])):
        for c, k in zip(cache, kept):
            c.view(torch.uint8).copy_(k)
        kv, keep = np.array(kv, np.int32), np.array(keep, np.int32)
        t[2].copy_(torch.from_numpy(kv))
        t[4].copy_(torch.from_numpy(keep))
        g.replay()
        torch.cuda.synchronize()
        plan = paged.evict(kv, keep, sc, tag, 4, base, slots)
        assert sum(len(m) for _, m in plan.values()) > 0
        check_evicted(S, kind, (S.Kp, S.Vp), before, plan, out, sc, tag, base, kv, keep)
    assert B.check_status() == 0


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_rows_that_should_move_without_a_page(B, kind):  # noqa: F811
    """Sources without a page, alone and beside others that come into the same page, and holes without one: what cannot be
    written stays, the rest moves, scores and positions follow the plan."""
    page, n_kv, hd = 16, 2, 64
    S = make(730, [(0, 400), (0, 250)], n_kv, n_kv, hd, page, kind)
    slots = S.table.shape[1] * page
    sc, tag, base = state(S, kind, 0, slots, False)
    sc[0, :, 32:48] -= 5.0                         # a page of holes alone
    sc[0, :, 64] -= 5.0                            # one hole, the rest of the page stays
    sc[0, :, 65:80] += 5.0
    sc[1, :, :120] -= 5.0                          # nothing of the first half stays
    keep = np.array([200, 120], np.int32)
    table = S.table.copy()
    table[0, [14, 17, 18, 22, 24]] = -1, S.P, -3, 1 << 30, -1     # some of the pages that rows leave
    table[0, 5] = -1                               # one that they enter
    table[1, 7:12] = -1
    plan = paged.evict(S.kv_len, keep, sc, tag, 0, base, slots)
    k0 = {"K": host(S.Kp), "V": host(S.Vp)}
    want = {n: c.copy() for n, c in k0.items()}
    e0 = {"K": S.Ke.copy(), "V": S.Ve.copy()} if kind == F8 else None
    e1 = {n: e.copy() for n, e in e0.items()} if kind == F8 else None
    here = lambda b, j: 0 <= table[b, j // page] < S.P      # noqa: E731
    lost = mixed = alone = 0
    for (b, g), (K, moves) in plan.items():
        holes = {d for d, _ in moves}
        for pg in sorted({d // page for d, _ in moves}):
            ins = [(d, s) for d, s in moves if d // page == pg and here(b, d) and here(b, s)]
            gone = sum(d // page == pg for d, _ in moves) - len(ins)
            lost, mixed, alone = lost + gone, mixed + (gone > 0 and len(ins) > 0), alone + (gone > 0 and here(b, pg * page) and not ins)
            if not ins:
                continue
            rest = [j for j in range(pg * page, min((pg + 1) * page, K)) if j not in holes]
            p = table[b, pg]
            for n in ("K", "V"):
                src = {s: k0[n][table[b, s // page], s % page, g] for _, s in ins}
                if kind != F8:
                    for d, s in ins:
                        want[n][p, d % page, g] = src[s]
                    continue
                es = {s: e0[n][table[b, s // page], g] for _, s in ins}
                now = max(list(es.values()) + ([e0[n][p, g]] if rest else []))
                for j in rest:
                    want[n][p, j % page, g] = paged.e4m3(k0[n][p, j % page, g] * 2.0 ** (e0[n][p, g] - now))
                for d, s in ins:
                    want[n][p, d % page, g] = paged.e4m3(src[s] * 2.0 ** (es[s] - now))
                e1[n][p, g] = now
    assert lost > 20 and mixed > 2 and alone > 2
    t = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, base, keep, table)]
    B.dllm_paged_evict(S.Kp, S.Vp, t[5], t[2], t[4], t[0], t[1], pos_base=t[3], K_scale=S.Ks, V_scale=S.Vs)
    assert B.check_status(reset=True) == B.STATUS_PAGE
    for n, pool in (("K", S.Kp), ("V", S.Vp)):
        assert np.array_equal(host(pool), want[n])
    if kind == F8:
        assert np.array_equal(exps(S.Ks), e1["K"]) and np.array_equal(exps(S.Vs), e1["V"])
    for (b, g), (K, moves) in plan.items():
        w, m = sc[b, g].copy(), tag[b, g].copy()
        for d, s in moves:
            w[d], m[d] = sc[b, g, s], tag[b, g, s]
        assert np.array_equal(t[0].cpu().numpy()[b, g, :K], w[:K]) and np.array_equal(t[1].cpu().numpy()[b, g, :K], m[:K])
    assert t[2].tolist() == keep.tolist() and t[3].tolist() == [base[0] + 200, base[1] + 130]


@pytest.mark.parametrize("page", [8, 32, 256])
def test_selections_past_shared_memory_over_8_bit_pages(B, page):  # noqa: F811
    """Keys, values and scales of every page, those of rows that stay and are rounded anew among them."""
    n_kv, hd, recent = 2, 64, 777
    S = make(740 + page, [(0, 60000), (0, 24577), (0, 25000)], n_kv, n_kv, hd, page, F8)
    slots = S.table.shape[1] * page
    sc, tag, base = state(S, F8, recent, slots, False)
    keep = np.array([41000, 24576, 3], np.int32)
    before = {"K": (S.Kc.copy(), S.Ke.copy()), "V": (S.Vc.copy(), S.Ve.copy())}
    t = [torch.from_numpy(x).cuda() for x in (sc, tag, S.kv_len, base, keep)]
    got = B.dllm_paged_evict(S.Kp, S.Vp, S.d[0], t[2], t[4], t[0], t[1], recent=recent, pos_base=t[3], K_scale=S.Ks, V_scale=S.Vs)
    assert B.check_status() == 0
    plan = paged.evict(S.kv_len, keep, sc, tag, recent, base, slots)
    grew = 0
    for n, pool, scale in (("K", S.Kp, S.Ks), ("V", S.Vp, S.Vs)):
        c0, e0 = before[n]
        want, e1 = c0.copy(), e0.copy()
        for (b, g), (K, moves) in plan.items():
            dst, src = (np.array([m[i] for m in moves], np.int64) for i in (0, 1))
            n_pg = -(-K // page)
            come, holes = np.full(n_pg, -1000), np.zeros(n_pg, np.int64)
            np.maximum.at(come, dst // page, e0[S.table[b, src // page], g])
            np.add.at(holes, dst // page, 1)
            rows = np.minimum(page, K - np.arange(n_pg) * page)
            p = S.table[b, :n_pg]
            now = np.where(holes == 0, e0[p, g], np.where(holes < rows, np.maximum(come, e0[p, g]), come))
            j = np.setdiff1d(np.arange(K), dst)
            j = j[now[j // page] > e0[p[j // page], g]]
            grew += len(j)
            at = p[j // page], j % page, g
            want[at] = paged.e4m3(c0[at] * 2.0 ** (e0[at[0], g] - now[j // page])[:, None])
            s = S.table[b, src // page]
            want[p[dst // page], dst % page, g] = paged.e4m3(c0[s, src % page, g] * 2.0 ** (e0[s, g] - now[dst // page])[:, None])
            e1[p, g] = now
        assert np.array_equal(exps(scale), e1) and np.array_equal(host(pool), want)
    assert grew > 1000
    for (b, g), (K, moves) in plan.items():
        w, m = sc[b, g].copy(), tag[b, g].copy()
        for d, s in moves:
            w[d], m[d] = sc[b, g, s], tag[b, g, s]
        assert np.array_equal(got[0].cpu().numpy()[b, g, :K], w[:K]) and np.array_equal(got[1].cpu().numpy()[b, g, :K], m[:K])
    assert got[2].tolist() == keep.tolist() and got[3].tolist() == (base + S.kv_len - keep).tolist()
