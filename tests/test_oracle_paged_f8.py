"""Closed forms of the oracle of the 8-bit pages, the key weights and the eviction, and their calls' refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_abi import dl  # noqa: F401  (the library fixture)


def test_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    fine = every[np.isfinite(every)]
    assert np.array_equal(paged.e4m3(fine), fine) and np.abs(fine).max() == 448
    s = np.unique(fine)
    for lo, hi in zip(s[:-1], s[1:]):                    # half way: to the even code; just beside it: to the nearer
        mid = (lo + hi) / 2
        a, b, c = paged.e4m3([mid, np.nextafter(mid, hi), np.nextafter(mid, lo)])
        assert b == hi and c == lo
        assert a == float(torch.tensor(mid, dtype=torch.float32).to(torch.float8_e4m3fn).float())
    assert paged.e4m3([1e9, -449.0]).tolist() == [448.0, -448.0] and np.isnan(paged.e4m3([np.nan]))[0]


def test_exponents_are_the_least_that_hold():
    assert [paged.exponent_for(x) for x in (0.0, 448.0, 449.0, 1.0, 1.75, 1.7500001, 2.0 ** 80)] == [-64, 0, 1, -8, -8, -7, 63]


def test_append_f8_scale_grows_and_stays():
    codes, e = np.zeros((2, 8, 1, 2)), np.zeros((2, 1), int)
    codes[1, :2, 0] = [[64.0, 3.0], [448.0, 0.0]]
    e[1] = -3
    table = np.array([[1, 0]])
    for top, want in ((10.0, -3), (500.0, 1)):
        x = np.array([[[top, 1.0]]])
        out, _, lost = paged.append_f8(x, x, codes, codes, e, e, table, [0, 1], [3])
        c, ex, wrote = out["K"]
        assert lost == 0 and ex[1, 0] == want and ex[0, 0] == 0
        np.testing.assert_allclose(c[1, :3, 0] * 2.0 ** want, [[8.0, 0.375], [56.0, 0.0], [top, 1.0]])
        assert wrote[1].tolist() == [want > -3] * 2 + [True] + [False] * 5 and not wrote[0].any()
    # a page that the rows fill from its first slot on forgets its scale
    out, _, _ = paged.append_f8(np.ones((1, 1, 2)), np.ones((1, 1, 2)), codes, codes, e + 40, e + 40, table, [0, 1], [9])
    assert out["V"][1][0, 0] == -8


def test_weights_of_a_softmax_sum_to_its_rows():
    g = synth.rng(71)
    Kp = g.standard_normal((3, 8, 1, 4))
    table, Q = np.array([[2, 0, 1]]), g.standard_normal((3, 2, 4))
    lse = paged.attention(Q, Kp, Kp, table, [0, 3], [19], mask_block=1)[2]
    sc, tag, _ = paged.weights(Q, Kp, table, [0, 3], [19], lse, np.full((1, 1, 20), 5.0), np.full((1, 1, 20), -7), 1,
                               pos_base=[100])
    assert np.allclose(sc[0, 0, :16].sum() - 16 * 5.0 + sc[0, 0, 16:19].sum(), 6.0) and sc[0, 0, 19] == 5.0
    assert tag[0, 0].tolist() == [-7] * 16 + [116, 117, 118] + [-7]
    assert (sc[0, 0, 16:19] < 6).all() and sc[0, 0, 18] < 2      # only the last row sees the last key


def test_evict_order_protection_and_ties():
    nan = np.nan
    sc = np.array([[[3.0, 1.0, nan, 1.0, 0.0, 9.0, -np.inf, 0.5]]])
    pos = np.array([[[0, 1, 2, 3, 4, 5, 6, 7]]])
    go = lambda keep, recent, base=None: paged.evict([8], [keep], sc, pos, recent, base, 8)[0, 0]   # noqa: E731
    assert go(3, 0) == (3, [(2, 5)])                     # 9, 3, and of the two ones the lower slot
    assert go(3, 2) == (3, [(0, 5), (1, 6), (2, 7)])     # slots 6 and 7 are protected, then 9
    assert go(1, 2) == (1, [(0, 7)])                     # not even all protected ones stay
    assert go(8, 0) == (8, []) and go(99, 0) == (8, []) and go(0, 3) == (0, []) and go(-4, 0) == (0, [])
    assert go(7, 0) == (7, [(2, 7)])                     # NaN goes before -inf
    assert go(3, 2, [6]) == go(3, 0)                     # positions below L + base - recent


def test_refusals_before_any_launch(dl):  # noqa: F811
    L = dl.lib()
    p, q, r, s = (C.c_void_p(x) for x in (256, 1 << 20, 1 << 21, 1 << 22))
    odd = C.c_void_p(264)

    def append(Q=p, K=p, V=p, st=(128, 128, 128), gq=None, gk=None, eps=1e-5, qs=p, kl=p, tab=p, mp=4, Qo=q, Kp=p, Vp=q,
               Ks=r, Vs=s, T=2, B=1, n_q=1, n_kv=1, hd=128, page=16, n_pages=4, idt=1):
        return L.dllm_paged_append_f8(Q, K, V, *st, gq, gk, eps, None, None, qs, kl, tab, mp, Qo, Kp, Vp, Ks, Vs, T, B, n_q,
                                      n_kv, hd, page, n_pages, idt, None)

    assert append(T=0) == 0
    assert append(K=None) == -1 and append(kl=None) == -1 and append(Vp=None) == -1 and append(Ks=None) == -1
    assert append(Vs=r) == -1 and append(Vp=p) == -1 and append(Qo=None) == -1 and append(Q=None, Qo=None, gq=p) == -1
    assert append(hd=96) == -2 and append(page=24) == -2 and append(B=1025) == -2
    assert append(B=0) == -1 and append(T=-1) == -1 and append(n_pages=0) == -1 and append(n_pages=1 << 28) == -1
    assert append(st=(128, 120, 128)) == -1 and append(st=(128, 132, 128)) == -1 and append(K=odd) == -1
    assert append(idt=2) == -1 and append(eps=-1.0) == -1 and append(gk=C.c_void_p(258)) == -1

    def append_at(base=p, T=0, Kp=p, dt=1):
        return L.dllm_paged_append_at(p, p, p, 128, 128, 128, None, None, 1e-5, None, base, p, p, p, 4, q, Kp, q, T, 1, 1, 1,
                                      128, 16, 4, dt, dt, None)

    assert append_at() == 0 and append_at(base=None) == 0 and append_at(T=2, Kp=None) == -1 and append_at(T=2, dt=2) == -1

    def attend(Q=p, st=128, Kp=p, Vp=q, Ks=r, Vs=s, tab=p, mp=4, mn=2, mb=0, sc=0.1, A=q, T=2, B=1, n_q=1, n_kv=1, hd=128,
               page=16, n_pages=4, ws=None, wb=0):
        return L.dllm_paged_attention_f8(Q, st, Kp, Vp, Ks, Vs, p, p, tab, mp, mn, mb, sc, A, None, T, B, n_q, n_kv, hd, page,
                                         n_pages, ws, wb, None)

    assert attend(T=0) == 0 and attend(mn=0) == 0
    assert attend(Q=None) == -1 and attend(A=None) == -1 and attend(A=p) == -1 and attend(Ks=None) == -1 and attend(Vs=None) == -1
    assert attend(n_q=3, n_kv=2) == -1 and attend(n_q=258, n_kv=2, st=258 * 128) == -2
    assert attend(sc=0.0) == -1 and attend(sc=float("inf")) == -1 and attend(mb=-1) == -1 and attend(mn=-1) == -1
    assert attend(hd=32) == -2 and attend(page=48) == -2 and attend(st=100) == -1 and attend(st=129) == -1
    need = L.dllm_paged_attention_f8_workspace_bytes(2, 1, 2, 1, 1, 128)
    assert attend() == -3 and need > 0 and attend(ws=p, wb=need - 1) == -3
    assert L.dllm_paged_attention_f8_workspace_bytes(2, 1, 2, 3, 2, 128) == 0

    def weigh(Q=p, st=128, Kp=p, Ks=None, mn=2, mb=0, sc=0.1, lse=p, score=r, out=q, slots=64, T=2, B=1, n_q=1, n_kv=1,
              hd=128, page=16, n_pages=4, dt=1):
        return L.dllm_paged_weights(Q, st, Kp, Ks, p, p, p, 4, mn, mb, sc, lse, None, score, out, None, slots, T, B, n_q, n_kv,
                                    hd, page, n_pages, dt, None)

    assert weigh(T=0) == 0 and weigh(mn=0) == 0
    assert weigh(Q=None) == -1 and weigh(lse=None) == -1 and weigh(score=None) == -1 and weigh(out=None) == -1
    assert weigh(dt=3) == -1 and weigh(dt=2) == -1 and weigh(Ks=r) == -1 and weigh(slots=0) == -1 and weigh(slots=(1 << 30) + 1) == -1
    assert weigh(n_q=3, n_kv=2) == -1 and weigh(hd=80) == -2 and weigh(st=64) == -1 and weigh(Q=odd) == -1
    assert weigh(B=1024, n_kv=32768, n_q=32768) == -1 and weigh(sc=-1.0) == -1

    def evict(Kp=p, Vp=q, Ks=None, Vs=None, kl=p, keep=p, recent=0, base=None, score=p, pos=p, slots=64, so=p, po=p, lo=p, bo=None,
              B=1, n_kv=1, hd=128, page=16, n_pages=4, dt=1, ws=p, wb=1 << 30):
        return L.dllm_paged_evict(Kp, Vp, Ks, Vs, kl, p, 4, keep, recent, base, score, pos, slots, so, po, lo, bo, B, n_kv, hd,
                                  page, n_pages, dt, ws, wb, None)

    assert evict(Kp=None) == -1 and evict(keep=None) == -1 and evict(pos=None) == -1 and evict(po=None) == -1 and evict(lo=None) == -1
    assert evict(score=None) == -1 and evict(so=None) == -1 and evict(Vp=p) == -1 and evict(recent=-1) == -1
    assert evict(base=p) == -1 and evict(bo=p) == -1 and evict(slots=0) == -1
    assert evict(dt=2) == -1 and evict(dt=2, Ks=r) == -1 and evict(dt=2, Ks=r, Vs=r) == -1 and evict(Ks=r, Vs=s) == -1
    assert evict(hd=72) == -2 and evict(page=4) == -2 and evict(B=1025) == -2
    need = L.dllm_paged_evict_workspace_bytes(1, 1, 64, 1)
    assert need > 0 and evict(wb=need - 1) == -3 and evict(ws=None) == -3
    assert L.dllm_paged_evict_workspace_bytes(1, 1, 64, 2) > need
    assert L.dllm_paged_evict_workspace_bytes(0, 1, 64, 1) == 0 and L.dllm_paged_evict_workspace_bytes(1, 1, (1 << 30) + 1, 1) == 0


def test_binding_refusals(dl):  # noqa: F811
    import torch
    f, i, u = torch.float32, torch.int32, torch.uint8
    codes = torch.zeros((2, 16, 1, 64), dtype=u).view(torch.float8_e4m3fn)
    exps = torch.zeros((2, 1), dtype=u).view(torch.float8_e8m0fnu)
    Kf = torch.zeros((2, 16, 1, 64), dtype=f)
    t, qs, kl = torch.zeros((1, 2), dtype=i), torch.zeros(2, dtype=i), torch.zeros(1, dtype=i)
    x, xb = torch.zeros((3, 1, 64), dtype=f), torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    sc, tag, lse = torch.zeros((1, 1, 32)), torch.zeros((1, 1, 32), dtype=i), torch.zeros((3, 1))
    calls = [
        lambda: dl.dllm_paged_append_f8(x, x, codes, codes.clone(), exps, exps.clone(), t, qs, kl),     # CPU tensors
        lambda: dl.dllm_paged_append_f8(x, x, Kf, Kf, exps, exps, t, qs, kl),                            # pages of fp32
        lambda: dl.dllm_paged_append_f8(x, x, codes, codes, exps[:1], exps, t, qs, kl),                  # scales' shape
        lambda: dl.dllm_paged_append(x, x, Kf, Kf.clone(), t, qs, kl, pos_base=torch.zeros(2, dtype=i)),
        lambda: dl.dllm_paged_attention_f8(xb, codes, codes, exps, exps, t, qs, kl, 3),
        lambda: dl.dllm_paged_attention_f8(x, codes, codes, exps, exps, t, qs, kl, 3),                   # Q of fp32
        lambda: dl.dllm_paged_attention_f8(xb, codes, codes, exps, None, t, qs, kl, 3),
        lambda: dl.dllm_paged_weights(x, Kf, t, qs, kl, 3, lse, sc),
        lambda: dl.dllm_paged_weights(x, codes, t, qs, kl, 3, lse, sc, K_scale=exps),                    # Q of fp32
        lambda: dl.dllm_paged_weights(xb, codes, t, qs, kl, 3, lse, sc),                                 # no scales
        lambda: dl.dllm_paged_weights(x, Kf, t, qs, kl, 3, lse, sc, K_scale=exps),
        lambda: dl.dllm_paged_weights(x, Kf, t, qs, kl, 3, lse[:2], sc),
        lambda: dl.dllm_paged_weights(x, Kf, t, qs, kl, 3, lse, sc, slot_pos=tag[..., :8]),
        lambda: dl.dllm_paged_weights(x, Kf, t, qs, kl, 3, lse, sc.double()),
        lambda: dl.dllm_paged_evict(Kf, Kf.clone(), t, kl, kl, sc, tag),
        lambda: dl.dllm_paged_evict(Kf, Kf.clone(), t, kl, kl, sc, tag, K_scale=exps, V_scale=exps),
        lambda: dl.dllm_paged_evict(codes, codes.clone(), t, kl, kl, sc, tag),
        lambda: dl.dllm_paged_evict(Kf, Kf.clone(), t, kl, qs, sc, tag),
        lambda: dl.dllm_paged_evict(Kf, Kf.clone(), t, kl, kl, sc, tag, pos_base=kl, out=(sc, tag, kl, None)),
        lambda: dl.dllm_paged_evict(Kf, Kf.clone(), t, kl, kl, sc, tag.float()),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(dl.DllmError):
            call()
            raise AssertionError(f"call {n} was taken")
