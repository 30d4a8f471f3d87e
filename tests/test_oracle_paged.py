"""Closed forms of the paged-operator oracle, and the operators' refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_abi import dl  # noqa: F401  (the library fixture)


def test_rows_know_their_sequence_and_position():
    r = paged.rows_of([0, 2, 2, 5], [7, 3, 2], 7)
    assert r.tolist() == [[0, 5], [0, 6], [2, -1], [2, 0], [2, 1], [-1, -1], [-1, -1]]


def test_append_norm_rotation_and_slot():
    Kp = np.zeros((3, 8, 1, 4))
    x = np.array([[[3.0, 0.0, 4.0, 0.0]]])
    table = np.array([[2, 0]])
    # position 9 of the second page (page 0, slot 1); norm of (3,0,4,0) is rms 2.5
    K, V, Q, lost = paged.append(x, x, Kp, Kp, table, [0, 1], [10], Q=x, Q_out=np.zeros((1, 1, 4)),
                                 gamma_k=np.ones(4), eps=0.0, inv_freq=np.array([np.pi / 18, 0.0]))
    assert lost == 0
    # pair (0, 2) turned by 9 * pi/18 = pi/2: (a, c) -> (-c, a)
    np.testing.assert_allclose(K[0, 1, 0], [-1.6, 0.0, 1.2, 0.0], atol=1e-12)
    np.testing.assert_allclose(Q[0, 0], [-4.0, 0.0, 3.0, 0.0], atol=1e-12)
    np.testing.assert_allclose(V[0, 1, 0], x[0, 0])
    assert np.count_nonzero(K) == 2 and np.count_nonzero(V) == 2


def test_attention_uniform_keys_average_the_visible_values():
    g = synth.rng(3)
    Kp, Vp = np.zeros((2, 8, 1, 4)), g.standard_normal((2, 8, 1, 4))
    table = np.array([[1, 0]])
    Q = g.standard_normal((3, 2, 4))
    A, Aa, lse, n = paged.attention(Q, Kp, Vp, table, [0, 3], [10], mask_block=1)
    V = np.concatenate([Vp[1], Vp[0]])[:, 0]
    assert n.tolist() == [8, 9, 10]
    for t in range(3):
        np.testing.assert_allclose(A[t, 1], V[:8 + t].mean(0), atol=1e-12)
        assert lse[t, 0] == pytest.approx(np.log(8 + t))
    A4, _, _, n4 = paged.attention(Q, Kp, Vp, table, [0, 3], [10], mask_block=4)
    assert n4.tolist() == [8, 10, 10]
    Ah, _, _, nh = paged.attention(Q, Kp, Vp, np.array([[-1, 0]]), [0, 3], [10])   # an absent page
    np.testing.assert_allclose(Ah[0, 0], V[8:10].mean(0), atol=1e-12)
    Z, _, l0, n0 = paged.attention(Q, Kp, Vp, np.array([[-1, 7]]), [0, 3], [10])
    assert not Z.any() and np.isneginf(l0).all() and not n0.any()


def test_sampling_order_filters_and_inverse():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3], np.float64)).astype(np.float32)
    assert [paged.sample_row(l, u)[0] for u in (0.0, 0.05, 0.15, 0.55, 0.75, 0.999)] == [0, 0, 1, 2, 3, 3]
    assert paged.sample_row(l, 0.0, top_k=2) == (1, pytest.approx(0.4 / 0.7))
    assert paged.sample_row(l, 0.6, top_k=2)[0] == 3
    assert paged.sample_row(l, 0.0, top_p=0.5)[0] == 1 and paged.sample_row(l, 0.99, top_p=0.5)[0] == 3
    assert paged.sample_row(l, 0.99, top_p=0.39)[0] == 1
    assert paged.sample_row(l, 0.0, min_p=0.6)[0] == 1 and paged.sample_row(l, 0.99, min_p=0.6)[0] == 3
    assert paged.sample_row(l, 0.99, temperature=0.0) == (1, 1.0)
    assert paged.sample_row([1.0, 1.0, 1.0, 0.0], 0.7, top_k=2)[0] == 1        # ties: lower ids
    assert paged.sample_row([np.nan, -np.inf, 0.0, np.nan], 0.5) == (2, 1.0)
    assert paged.sample_row([np.nan, -np.inf], 0.5) == (-1, 0.0)
    assert paged.sample_row([np.inf, 1.0, np.inf], 0.7)[0] == 2


def test_refusals_before_any_launch(dl):  # noqa: F811
    L = dl.lib()
    p, q = C.c_void_p(256), C.c_void_p(1 << 20)

    def append(Q=p, K=p, V=p, st=(128, 128, 128), gq=None, gk=None, eps=1e-5, freq=None, qs=p, kl=p, tab=p, mp=4,
               Qo=q, Kp=p, Vp=q, T=2, B=1, n_q=1, n_kv=1, hd=128, page=16, n_pages=4, idt=1, dt=1):
        return L.dllm_paged_append(Q, K, V, *st, gq, gk, eps, freq, qs, kl, tab, mp, Qo, Kp, Vp, T, B, n_q, n_kv, hd,
                                   page, n_pages, idt, dt, None)

    assert append(T=0) == 0
    assert append(K=None) == -1 and append(qs=None) == -1 and append(Kp=None) == -1
    assert append(Qo=None) == -1 and append(Q=None) == -1 and append(Q=None, Qo=None, gq=p) == -1
    assert append(hd=96) == -2 and append(page=24) == -2 and append(page=4) == -2 and append(page=512) == -2
    assert append(B=1025) == -2
    assert append(B=0) == -1 and append(T=-1) == -1 and append(n_pages=0) == -1 and append(mp=0) == -1
    assert append(st=(128, 120, 128)) == -1 and append(st=(128, 132, 128)) == -1       # overlap, alignment
    assert append(K=C.c_void_p(264)) == -1 and append(gk=C.c_void_p(258)) == -1
    assert append(idt=1, dt=0) == -1 and append(idt=2) == -1
    assert append(n_pages=1 << 28) == -1 and append(mp=1 << 28) == -1                  # past the int range
    assert append(Vp=p) == -1 and append(eps=-1.0) == -1

    def attend(Q=p, st=128, Kp=p, Vp=q, qs=p, kl=p, tab=p, mp=4, mn=2, mb=0, sc=0.1, A=q, T=2, B=1, n_q=1, n_kv=1, hd=128,
               page=16, n_pages=4, dt=1, ws=None, wb=0):
        return L.dllm_paged_attention(Q, st, Kp, Vp, qs, kl, tab, mp, mn, mb, sc, A, None, T, B, n_q, n_kv, hd, page,
                                      n_pages, dt, ws, wb, None)

    assert attend(T=0) == 0 and attend(mn=0) == 0
    assert attend(Q=None) == -1 and attend(A=None) == -1 and attend(A=p) == -1 and attend(tab=None) == -1
    assert attend(n_q=3, n_kv=2) == -1 and attend(n_q=129 * 2, n_kv=2, st=129 * 2 * 128) == -2
    assert attend(sc=0.0) == -1 and attend(sc=float("nan")) == -1 and attend(mb=-1) == -1 and attend(mn=-1) == -1
    assert attend(hd=32) == -2 and attend(page=48) == -2 and attend(st=100) == -1 and attend(st=129) == -1
    assert attend(T=1 << 24, n_q=128, st=128 * 128) == -1                               # T * n_q past 2^30
    need = L.dllm_paged_attention_workspace_bytes(2, 1, 2, 1, 1, 128, 1)
    if need:
        assert attend(ws=p, wb=need - 1) == -3 and attend() == -3
    assert L.dllm_paged_attention_workspace_bytes(0, 1, 2, 1, 1, 128, 1) == 0

    def sample(l=p, u=p, tok=p, pr=p, B=1, M=2, V=100, dt=0, ws=p, wb=1 << 20):
        return L.dllm_sample(l, u, None, None, None, None, None, tok, pr, B, M, V, dt, ws, wb, None)

    assert sample(B=0) == 0 and sample(M=0) == 0
    assert sample(l=None) == -1 and sample(u=None) == -1 and sample(tok=None) == -1 and sample(pr=None) == -1
    assert sample(V=0) == -1 and sample(V=262145) == -2 and sample(dt=2) == -1
    assert sample(B=1 << 20, M=1 << 20) == -1 and sample(l=C.c_void_p(258)) == -1
    assert sample(B=(1 << 24) + 1, M=1) == -1 and L.dllm_sample_workspace_bytes((1 << 24) + 1, 1, 100) == 0
    need = L.dllm_sample_workspace_bytes(1, 2, 100)
    assert need > 0 and sample(wb=need - 1) == -3 and sample(ws=None) == -3


def test_binding_refusals(dl):  # noqa: F811
    import torch
    f, i = torch.float32, torch.int32
    Kp = torch.zeros((2, 16, 1, 64), dtype=f)
    t, qs, kl = torch.zeros((1, 2), dtype=i), torch.zeros(2, dtype=i), torch.zeros(1, dtype=i)
    x = torch.zeros((3, 1, 64), dtype=f)
    with pytest.raises(dl.DllmError):      # CPU tensors
        dl.dllm_paged_append(x, x, Kp, Kp, t, qs, kl)
    with pytest.raises(dl.DllmError):
        dl.dllm_paged_attention(x, Kp, Kp, t, qs, kl, 3)
    with pytest.raises(dl.DllmError):      # q_start of the wrong length
        dl.dllm_paged_attention(x, Kp, Kp, t, kl, kl, 3)
    with pytest.raises(dl.DllmError):
        dl.dllm_sample(torch.zeros((1, 1, 8)), torch.zeros((1, 1)))
    with pytest.raises(dl.DllmError):
        dl.dllm_sample(torch.zeros((1, 1, 8)), torch.zeros((1, 2)))
