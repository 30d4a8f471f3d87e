"""Masks in blocks over a cache that gives up slots: as long as their number is a multiple of the block, a row sees the
tokens of the blocks up to its own, wherever their keys have moved."""
import numpy as np
import pytest

from oracle import paged
from test_gpu_paged import F32, B, dev, host  # noqa: F401  (B: the library fixture)
from test_gpu_paged_evict import F8, IDS, KINDS, make
from test_gpu_paged_f8 import exps

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_blocks_stay_those_of_the_tokens(B, kind):  # noqa: F811
    n_q, n_kv, hd, page, m = 4, 2, 64, 16, 8
    S = make(770, [(0, 240), (0, 240)], n_q, n_kv, hd, page, kind)
    slots = S.table.shape[1] * page
    f = (10000.0 ** (-2 * np.arange(hd // 2) / hd)).astype(np.float32)
    score = torch.zeros((2, n_kv, slots), device="cuda")
    tags = torch.zeros((2, n_kv, slots), dtype=torch.int32, device="cuda")
    kv, base = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2))
    # prompts, whole blocks, rows that begin and end inside a block; the keys that stay: L - K = 64, 24, 0, 40, 16, 8
    for new, gone in (([120, 101], [64, 24]), ([24, 16], [0, 40]), ([21, 3], [16, 0]), ([3, 30], [8, 8]), ([1, 1], [0, 0]), ([40, 7], [0, 0])):
        st = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        qs, T, most = torch.from_numpy(st).cuda(), int(sum(new)), max(new)
        kv += torch.tensor(new, dtype=torch.int32, device="cuda")
        qkv = dev(S.g.standard_normal((T, n_q + 2 * n_kv, hd), dtype=np.float32), S.qdt)
        Q, K, V = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        lse = torch.empty((T, n_q), device="cuda")
        kw = dict(Q=Q, inv_freq=torch.from_numpy(f).cuda(), pos_base=base)
        if kind == F8:
            pool = (S.Kp, S.Vp, S.Ks, S.Vs)
            q = B.dllm_paged_append_f8(K, V, *pool, S.d[0], qs, kv, **kw)
            A = B.dllm_paged_attention_f8(q, *pool, S.d[0], qs, kv, most, mask_block=m, lse=lse)
            Kv, Vv = (host(c) * 2.0 ** exps(s)[:, None, :, None] for c, s in ((S.Kp, S.Ks), (S.Vp, S.Vs)))
        else:
            q = B.dllm_paged_append(K, V, S.Kp, S.Vp, S.d[0], qs, kv, **kw)
            A = B.dllm_paged_attention(q, S.Kp, S.Vp, S.d[0], qs, kv, most, mask_block=m, lse=lse)
            Kv, Vv = host(S.Kp), host(S.Vp)
        B.dllm_paged_weights(q, S.Kp, S.d[0], qs, kv, most, lse, score, slot_pos=tags, K_scale=S.Ks, mask_block=m, pos_base=base)
        qh, tag, lens, bases = host(q), tags.cpu().numpy(), kv.tolist(), base.tolist()
        for t, (b, p) in enumerate(paged.rows_of(st, kv.cpu().numpy(), T)):
            j = np.arange(lens[b])
            at = S.table[b, j // page], j % page
            for h in range(n_q):
                g = h // (n_q // n_kv)
                seen = tag[b, g, :lens[b]] // m <= (p + bases[b]) // m        # by the tokens' positions
                s = np.where(seen, Kv[at[0], at[1], g] @ qh[t, h] * hd ** -0.5, -np.inf)
                w = np.exp(s - s.max())
                ref = (w / w.sum()) @ Vv[at[0], at[1], g]
                tol = 1e-4 if kind == F32 else 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2e-3) * ((w / w.sum()) @ np.abs(Vv[at[0], at[1], g]))
                assert (np.abs(host(A[t, h]) - ref) <= tol).all(), (t, h)
        keep = kv - torch.tensor(gone, dtype=torch.int32, device="cuda")
        B.dllm_paged_evict(S.Kp, S.Vp, S.d[0], kv, keep, score, tags, recent=m, pos_base=base, K_scale=S.Ks, V_scale=S.Vs)
    assert B.check_status() == 0 and base.tolist() == [88, 72]
