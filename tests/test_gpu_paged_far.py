"""The paged operators and the sampling where offsets pass 32 bits: pools of 2^33 elements, of which only a few pages
are used, and logits of more than 2^32.  Tolerances as in the parity tests."""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_gpu_paged import B, BF, F32, U, check_attention, dev, host  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class _S:
    pass


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_pages_at_the_far_end_of_a_large_pool(B, dt):  # noqa: F811
    n_pages, page, n_kv, hd, n_q = 1 << 17, 64, 8, 128, 16
    Kp, Vp = (torch.empty((n_pages, page, n_kv, hd), dtype=dt, device="cuda") for _ in range(2))
    assert Kp.numel() == 1 << 33
    g = synth.rng(91)
    seqs = [(5, 200), (64, 64), (1, 300)]
    ids = np.array([n_pages - 1, 3, n_pages - 2, (1 << 16) + 1, 0, (1 << 15) - 1, n_pages // 2, 7, n_pages - 9, 100000], np.int32)
    table = np.full((3, 5), -1, np.int32)
    table[0, :4], table[1, :1], table[2] = ids[:4], ids[4:5], ids[5:]
    small = {int(p): i for i, p in enumerate(ids)}
    K0, V0 = (dev(g.standard_normal((len(ids), page, n_kv, hd), dtype=np.float32), dt) for _ in range(2))
    at = torch.from_numpy(ids.astype(np.int64)).cuda()
    Kp[at], Vp[at] = K0, V0
    st, kv = np.array([0, 5, 69, 70], np.int32), np.array([k for _, k in seqs], np.int32)
    d = [torch.from_numpy(a).cuda() for a in (table, st, kv)]
    Q, K, V = (dev(g.standard_normal((70, h, hd), dtype=np.float32), dt) for h in (n_q, n_kv, n_kv))
    Qo = B.dllm_paged_append(K, V, Kp, Vp, *d, Q=Q)
    near = np.vectorize(lambda p: small.get(int(p), -1))(table)                  # the same pages in a small pool
    Kr, Vr, _, lost = paged.append(host(K), host(V), host(K0), host(V0), near, st, kv)
    assert lost == 0 and torch.equal(Qo, Q)
    assert np.array_equal(host(Kp[at]), Kr) and np.array_equal(host(Vp[at]), Vr)
    S = _S()
    S.T, S.rows, S.P, S.hd, S.Q, S.Kp = 70, 70, len(ids), hd, Q, Kp[at]
    lse = torch.empty((70, n_q), device="cuda")
    A = B.dllm_paged_attention(Q, Kp, Vp, *d, 64, mask_block=1, lse=lse)
    check_attention(A, lse, paged.attention(host(Q), Kr, Vr, near, st, kv, 1), S, dt)
    assert B.check_status() == 0


@pytest.mark.parametrize("V,rows", [(4096, 1100000), (200003, 21600)])
def test_rows_past_32_bits_of_logits(B, V, rows):  # noqa: F811
    l = torch.zeros((1, rows, V), dtype=BF, device="cuda")
    assert l.numel() > 1 << 32
    g = synth.rng(92)
    u = torch.from_numpy(g.random((1, rows)).astype(np.float32)).cuda()
    look = [0, rows // 2, rows - 2, rows - 1]
    for i in look:
        l[0, i] = dev(g.standard_normal(V, dtype=np.float32) * 3, BF)
    p = torch.tensor([0.9], device="cuda")
    tok, prob = B.dllm_sample(l, u, top_p=p, top_k=torch.tensor([300], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for i in look:
        rt, rp = paged.sample_row(host(l[0, i]), float(u[0, i]), 1.0, 300, 0.9)
        assert int(tok[0, i]) == rt and float(prob[0, i]) == pytest.approx(rp, rel=2.0 ** -24 + 1e-9)
    # the others: 300 equal weights, of which 0.9 stay
    same = torch.ones(rows, dtype=torch.bool, device="cuda")
    same[look] = False
    assert (prob[0][same] == prob[0, 1]).all() and (tok[0][same] < 270).all() and (tok[0] >= 0).all()
    assert float(prob[0, 1]) == pytest.approx(1 / 270, rel=2.0 ** -24 + 1e-9)
    assert B.check_status() == 0
