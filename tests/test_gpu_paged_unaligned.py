"""Scores, positions and log-sum-exps of the key weights and the eviction start anywhere: the header asks only
pages and rows of queries to be aligned."""
import ctypes as C

import numpy as np
import pytest

from test_abi import dl  # noqa: F401  (the library fixture)

torch = pytest.importorskip("torch")


def test_the_library_takes_unaligned_scores(dl):  # noqa: F811
    """No GPU: without rows there is nothing to launch, and the arguments have been looked at."""
    L = dl.lib()
    buf = (C.c_char * 4096)()
    p = (C.addressof(buf) + 255) & ~255

    def weigh(K=p, score=p + 260, T=0):
        return L.dllm_paged_weights(p, 128, K, None, p, p, p, 4, 2, 0, 0.1, p, None, score, score, None, 64, T, 1, 1, 1, 128, 16, 4, 1, None)

    assert weigh() == 0 and weigh(score=p) == 0
    assert weigh(K=p + 4) == -1 and weigh(score=None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "f8"])
def test_results_do_not_depend_on_where_arrays_start(dl, kind):  # noqa: F811
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_paged import BF, F32, dev
    from test_gpu_paged_evict import F8, make
    k = {"bf16": BF, "f32": F32, "f8": F8}[kind]
    seqs = [(3, 300), (1, 77), (40, 130)]
    S = make(760, seqs, 4, 2, 64, 16, k)
    Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), S.qdt)
    slots = S.table.shape[1] * 16 + 1
    sc = torch.from_numpy(S.g.random((3, 2, slots)).astype(np.float32)).cuda()
    lse = torch.from_numpy(S.g.random((S.T, 4)).astype(np.float32) + 5).cuda()
    keep = torch.tensor([200, 70, 9], dtype=torch.int32, device="cuda")
    pool = [t.view(torch.uint8).clone() for t in (S.Kp, S.Vp)]
    scales = [] if k is not F8 else [t.view(torch.uint8).clone() for t in (S.Ks, S.Vs)]
    got = []
    for shift in (0, 1, 3):
        at = lambda t: torch.cat([t.new_zeros(shift), t.reshape(-1)])[shift:].view(t.shape)   # noqa: E731
        score, l, tags, kv = at(sc), at(lse), at(torch.zeros_like(sc, dtype=torch.int32)), at(S.d[2])
        assert score.data_ptr() % 16 == 4 * shift
        for t, c in zip((S.Kp, S.Vp), pool):
            t.view(torch.uint8).copy_(c)
        for t, c in zip((S.Ks, S.Vs), scales):
            t.view(torch.uint8).copy_(c)
        dl.dllm_paged_weights(Q, S.Kp, *S.d, 40, l, score, slot_pos=tags, K_scale=S.Ks, mask_block=1)
        weighed = score.clone()
        dl.dllm_paged_evict(S.Kp, S.Vp, S.d[0], kv, at(keep), score, tags, recent=5, K_scale=S.Ks, V_scale=S.Vs)
        got.append([weighed, score, tags, kv, S.Kp.view(torch.uint8).clone(), S.Vp.view(torch.uint8).clone()])
    assert dl.check_status() == 0 and got[0][3].tolist() == [200, 70, 9]
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
