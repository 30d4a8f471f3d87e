"""The 8-bit pages, key weights and eviction where the parity tests' sizes do not reach: many key tiles for every CTA,
selections past what shared memory holds, pools past 32 bits, other streams and threads.  Tolerances as in the parity
tests (test_gpu_paged_f8.py, test_gpu_paged_evict.py)."""
import threading

import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_gpu_paged import BF, F32, B, Batch, dev, host  # noqa: F401  (B: the library fixture)
from test_gpu_paged_f8 import E4M3, E8M0, Batch8, exps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dense64(S, kind, b, n):
    """Keys of sequence b, fp64 on the device."""
    ids = S.d[0][b, :-(-n // S.page)].long()
    K = S.Kp[ids].double()
    if kind == "f8":
        K = K * torch.exp2(S.Ks.view(torch.uint8)[ids].double() - 127)[:, None, :, None]
    return K.reshape(-1, S.n_kv, S.hd)[:n]


def weigh_and_check(B, S, kind, n_q, most, slots, repeat):  # noqa: F811
    """Causal weights of a batch, three times into other arrays, with the lse of exact scores."""
    n_kv, hd, G = S.n_kv, S.hd, n_q // S.n_kv
    nb = len(S.seqs)
    Q = dev(S.g.standard_normal((S.T, n_q, hd), dtype=np.float32), BF)
    sc = torch.rand((nb, n_kv, slots), device="cuda")
    tag = torch.full((nb, n_kv, slots), -5, dtype=torch.int32, device="cuda")
    lse = torch.empty((S.T, n_q), device="cuda")
    for b, (n, k) in enumerate(S.seqs):
        if n == 0:
            continue
        r0 = int(S.q_start[b])
        s = torch.einsum("thd,jhd->thj", Q[r0:r0 + n].double(), dense64(S, kind, b, k).repeat_interleave(G, 1)) / hd ** 0.5
        seen = (torch.arange(k, device="cuda")[None] <= torch.arange(k - n, k, device="cuda")[:, None])[:, None]
        lse[r0:r0 + n] = torch.where(seen, s, -torch.inf).logsumexp(-1).float()
    out = torch.full_like(sc, 77.0)
    for _ in range(repeat):
        B.dllm_paged_weights(Q, S.Kp, *S.d, most, lse, sc, slot_pos=tag, K_scale=S.Ks if kind == "f8" else None, mask_block=1,
                             score_out=out)
    for b, (n, k) in enumerate(S.seqs):
        if n == 0:
            assert (out[b] == 77).all() and (tag[b] == -5).all()
            continue
        r0 = int(S.q_start[b])
        q, l = Q[r0:r0 + n].double(), lse[r0:r0 + n].double()
        keys = dense64(S, kind, b, k)
        s = torch.einsum("thd,jhd->thj", q, keys.repeat_interleave(G, 1)) / hd ** 0.5
        seen = (torch.arange(k, device="cuda")[None] <= torch.arange(k - n, k, device="cuda")[:, None])[:, None]
        w = torch.where(seen, torch.exp(s - l[..., None]), 0.0)
        fold = lambda x: x.reshape(n, n_kv, G, k).sum((0, 2))   # noqa: E731
        want, mag = fold(w), fold(w * (1 + s.abs() + l.abs()[..., None]))
        first = k - n
        want[:, :first] += sc[b, :, :first]
        mag[:, :first] += sc[b, :, :first]
        # hd 2^-23 |q| |k| scale of a score, its product with log2 e, the exponential, n additions
        qk = q.norm(dim=-1).max() * keys.norm(dim=-1).max() / hd ** 0.5
        tol = mag * (hd * 2.0 ** -23 * float(qk) + 2.0 ** -20 + n * G * 2.0 ** -24)
        assert ((out[b, :, :k].double() - want).abs() <= tol + 1e-30).all(), b
        assert (out[b, :, k:] == 77).all()
        assert (tag[b, :, first:k] == torch.arange(first, k, device="cuda")).all() and (tag[b, :, :first] == -5).all()
    assert B.check_status() == 0


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("kind", [BF, "f8"], ids=["bf16", "f8"])
def test_weights_over_many_tiles(B, kind, new):  # noqa: F811
    """Some 30 tiles of 128 keys a CTA: every ring goes round."""
    lens = [8000, 7999, 8129, 300, 6500, 7000, 129, 5000, 8192, 4097, 8000, 3333, 7777, 6400, 8191, 2048]
    seqs = [(max(0, new - (i % 3)), n) for i, n in enumerate(lens)]
    S = Batch8(660, seqs, 28, 4, 128, 16, spread=2) if kind == "f8" else Batch(660, seqs, 28, 4, 128, 16, kind)
    weigh_and_check(B, S, kind, 28, new, 8192, 3)


@pytest.mark.parametrize("new", [1, 4, 40])
@pytest.mark.parametrize("kind", [BF, "f8"], ids=["bf16", "f8"])
def test_weights_of_many_short_sequences(B, kind, new):  # noqa: F811
    """1024 sequences of one to three tiles a head: queries change with nearly every tile, in one row tile and in more."""
    g = synth.rng(661)
    seqs = [(int(g.integers(0, new + 1)), 0) for _ in range(1024)]
    seqs = [(n, n + int(g.integers(0, 300 if b % 5 == 0 else 100))) for b, (n, _) in enumerate(seqs)]
    S = Batch8(662, seqs, 8, 2, 64, 8, spread=2) if kind == "f8" else Batch(662, seqs, 8, 2, 64, 8, kind)
    weigh_and_check(B, S, kind, 8, new, 344, 2)


@pytest.mark.parametrize("kind", [F32, "f8"], ids=["f32", "f8"])
@pytest.mark.parametrize("levels", [0, 3])
def test_evict_selects_past_shared_memory(B, levels, kind):  # noqa: F811
    """60,000 slots a head, scores that differ or of three values, protected ones spread over all slots."""
    L, K, recent, page, n_kv, hd = 60000, 41000, 777, 16, 2, 64
    seqs = [(0, L), (0, 24577), (0, 25000)]
    S = Batch8(670, seqs, 2, n_kv, hd, page, spread=2) if kind == "f8" else Batch(670, seqs, 2, n_kv, hd, page, kind)
    g = S.g
    slots = S.table.shape[1] * page
    sc = g.random((3, n_kv, slots)).astype(np.float32)
    if levels:
        sc = np.floor(sc * levels).astype(np.float32)
    tag = np.stack([np.stack([g.permutation(slots) for _ in range(n_kv)]) for _ in range(3)]).astype(np.int32)
    keep, kv, base = np.array([K, 24576, 3], np.int32), S.kv_len, np.array([0, 5, 100], np.int32)
    k0, v0 = host(S.Kp), host(S.Vp)
    if kind == "f8":
        e0 = exps(S.Ks)
    t = [torch.from_numpy(a).cuda() for a in (kv, keep, sc, tag, base)]
    d = [torch.from_numpy(a).cuda() for a in (S.table,)]
    out = [torch.full_like(t[2], -1.0), torch.full_like(t[3], -1), torch.empty_like(t[0]), torch.empty_like(t[4])]
    B.dllm_paged_evict(S.Kp, S.Vp, d[0], t[0], t[1], t[2], t[3], recent=recent, pos_base=t[4], out=out,
                       K_scale=S.Ks if kind == "f8" else None, V_scale=S.Vs if kind == "f8" else None)
    plan = paged.evict(kv, keep, sc, tag, recent, base, slots)
    k1, v1, so, to = host(S.Kp), host(S.Vp), out[0].cpu().numpy(), out[1].cpu().numpy()
    assert out[2].tolist() == keep.tolist() and out[3].tolist() == [L - K, 6, 25097]
    if kind == "f8":
        e1 = exps(S.Ks)
    for (b, h), (n, moves) in plan.items():
        w, m = sc[b, h].copy(), tag[b, h].copy()
        dst, src = (np.array([x[i] for x in moves], np.int64) for i in (0, 1))
        w[dst], m[dst] = sc[b, h, src], tag[b, h, src]
        assert np.array_equal(so[b, h, :n], w[:n]) and np.array_equal(to[b, h, :n], m[:n])
        pd, ps = S.table[b, dst // page], S.table[b, src // page]
        if kind == "f8":
            scale = 2.0 ** (e0[ps, h] - e1[pd, h])
            assert (scale <= 1).all()
            assert np.array_equal(k1[pd, dst % page, h], paged.e4m3(k0[ps, src % page, h] * scale[:, None]))
        else:
            assert np.array_equal(k1[pd, dst % page, h], k0[ps, src % page, h])
            assert np.array_equal(v1[pd, dst % page, h], v0[ps, src % page, h])
    assert B.check_status() == 0


def test_smaller_cache_at_the_far_end_of_a_large_pool(B):  # noqa: F811
    n_pages, page, n_kv, hd, n_q = 1 << 17, 64, 8, 128, 16
    Kp, Vp = (torch.zeros((n_pages, page, n_kv, hd), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    assert Kp.numel() == 1 << 33
    Ks, Vs = (torch.full((n_pages, n_kv), 127, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))
    g = synth.rng(680)
    ids = np.array([n_pages - 1, 3, n_pages - 2, (1 << 16) + 1, 0, (1 << 15) - 1, n_pages // 2, 7, n_pages - 9, 100000], np.int32)
    table = np.full((3, 5), -1, np.int32)
    table[0, :4], table[1, :1], table[2] = ids[:4], ids[4:5], ids[5:]
    small = {int(p): i for i, p in enumerate(ids)}
    near = np.vectorize(lambda p: small.get(int(p), -1))(table).astype(np.int32)   # the same pages in a small pool
    at = torch.from_numpy(ids.astype(np.int64)).cuda()
    kv, n = np.array([200, 64, 300], np.int32), np.array([200, 64, 300])
    st = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    Q, K, V = (dev(g.standard_normal((564, h, hd), dtype=np.float32), BF) for h in (n_q, n_kv, n_kv))
    results = []
    for pool, tab in (((Kp, Vp, Ks, Vs), table), (tuple(x.view(torch.uint8)[at].view(x.dtype) for x in (Kp, Vp, Ks, Vs)), near)):
        d = [torch.from_numpy(a).cuda() for a in (tab, st, kv)]
        sc = torch.zeros((3, n_kv, 320), device="cuda")
        tag = torch.zeros((3, n_kv, 320), dtype=torch.int32, device="cuda")
        lens, keep = d[2].clone(), torch.tensor([90, 64, 70], dtype=torch.int32, device="cuda")
        lse = torch.empty((564, n_q), device="cuda")
        B.dllm_paged_append_f8(K, V, *pool, *d)
        A = B.dllm_paged_attention_f8(Q, *pool, *d, 300, mask_block=1, lse=lse)
        B.dllm_paged_weights(Q, pool[0], *d, 300, lse, sc, slot_pos=tag, K_scale=pool[2], mask_block=1)
        total = sc.sum((1, 2))
        B.dllm_paged_evict(pool[0], pool[1], d[0], lens, keep, sc, tag, recent=16, K_scale=pool[2], V_scale=pool[3])
        mine = [x.view(torch.uint8)[at] if pool[0] is Kp else x.view(torch.uint8) for x in pool]
        results.append([A, lse, sc, tag, lens, *mine])
        assert torch.allclose(total.cpu(), torch.from_numpy(n * n_q).float(), rtol=1e-3)
    assert all(torch.equal(a, b) for a, b in zip(*results)) and B.check_status() == 0


def server(B, S, seed):  # noqa: F811
    """A chain of all four calls over its own copies of the cache -> its outputs."""
    g = synth.rng(seed)
    n_q, n_kv, hd = 8, 2, 128
    Q, K, V = (dev(g.standard_normal((S.T, h, hd), dtype=np.float32), BF) for h in (n_q, n_kv, n_kv))
    most = max(n for n, _ in S.seqs)
    slots = S.table.shape[1] * S.page
    keep = torch.tensor([max(1, k // 2) for _, k in S.seqs], dtype=torch.int32, device="cuda")
    lse0 = torch.empty((S.T, n_q), device="cuda")

    def run():
        pool = [x.clone() for x in (S.Kp, S.Vp)] + [x.view(torch.uint8).clone().view(E8M0) for x in (S.Ks, S.Vs)]
        sc = torch.zeros((len(S.seqs), n_kv, slots), device="cuda")
        tag = torch.zeros((len(S.seqs), n_kv, slots), dtype=torch.int32, device="cuda")
        kv, lse = S.d[2].clone(), torch.empty_like(lse0)
        B.dllm_paged_append_f8(K, V, *pool, *S.d)
        A = B.dllm_paged_attention_f8(Q, *pool, *S.d, most, mask_block=1, lse=lse)
        B.dllm_paged_weights(Q, pool[0], *S.d, most, lse, sc, slot_pos=tag, K_scale=pool[2], mask_block=1)
        B.dllm_paged_evict(pool[0], pool[1], S.d[0], kv, keep, sc, tag, recent=8, K_scale=pool[2], V_scale=pool[3])
        return A, lse, sc, tag, kv, *(x.view(torch.uint8) for x in pool)
    return run


SERVED = [[(1, 3000)] * 9, [(200, 900), (64, 2000), (5, 9000)]]


def test_another_stream_and_two_graphs(B):  # noqa: F811
    """The chain on a side stream behind work that it depends on, and two captured chains replayed in turn."""
    runs = [server(B, Batch8(690 + i, q, 8, 2, 128, 32, spread=1), 695 + i) for i, q in enumerate(SERVED)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
        got = [r() for r in runs]
    side.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, got) for a, b in zip(w, o))
    graphs, outs = [], []
    for r in runs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(r())
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, o in zip(want, outs) for a, b in zip(w, o))
    assert B.check_status() == 0


def test_threads_on_one_stream(B):  # noqa: F811
    runs = [server(B, Batch8(690 + i, q, 8, 2, 128, 32, spread=1), 695 + i) for i, q in enumerate(SERVED)]
    pairs = [(r, r()) for r in runs]
    torch.cuda.synchronize()
    start, right, wrong = threading.Barrier(2), [], []

    def work(run, want):
        start.wait(30)
        for _ in range(20):
            outs = [run() for _ in range(2)]
            for got in outs:
                (right if all(torch.equal(g, w) for g, w in zip(got, want)) else wrong).append(1)

    threads = [threading.Thread(target=work, args=p) for p in pairs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len(right) == 2 * 20 * 2 and B.check_status() == 0
