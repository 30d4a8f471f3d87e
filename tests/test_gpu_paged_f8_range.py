"""GPU parity of the attention over 8-bit pages whose value scales are at both ends of their range, with
the tolerances of test_gpu_paged_f8.py.
"""
import numpy as np
import pytest

from oracle import paged
from test_gpu_paged import BF, B, dev  # noqa: F401  (B: the library fixture)
from test_gpu_paged_f8 import Batch8, check_attention

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# (new rows, keys), n_q, n_kv, hd, page, mask_block: the forms of up to 8, 16, 32, 64 and 128 rows of a key head
FORMS = [
    ([(1, 16000), (2, 777)], 4, 1, 128, 16, 0),
    ([(4, 9001), (1, 130)], 6, 2, 64, 64, 1),
    ([(30, 5000)], 1, 1, 128, 256, 0),
    ([(33, 4100), (7, 300)], 2, 2, 64, 8, 4),
    ([(40, 6000), (130, 1100)], 2, 1, 128, 32, 1),
]


def attend(B, S, mb, scale):  # noqa: F811
    lse = torch.empty((S.T, S.n_q), device="cuda")
    A = B.dllm_paged_attention_f8(S.Q, *S.cache(), max(n for n, _ in S.seqs), mask_block=mb, scale=scale, lse=lse)
    assert B.check_status() == 0
    return A, lse


def with_scores(i, offset, spread=0):
    """Scores of N(0, 1) plus offset(b, j) times the row's first element: a Batch8 whose keys hold that offset in dim 0."""
    seqs, n_q, n_kv, hd, page, mb = FORMS[i]
    S = Batch8(900 + i, seqs, n_q, n_kv, hd, page, spread=spread)
    S.Ke[...] = -7
    S.Kc[..., 0] = 0
    for b, (_, k) in enumerate(seqs):
        j = np.arange(k)
        S.Kc[S.table[b, j // page], j % page, :, 0] = paged.e4m3(offset(b, j, k) * 128)[:, None]
    S.upload()
    S.poison()
    S.Q = S.g.standard_normal((S.T, n_q, hd)).astype(np.float32) * 1.28 / hd ** 0.5
    return S, mb


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_values_at_both_ends_of_the_scales(B, i, late):  # noqa: F811
    """Pages of zeros (scale 2^-64) beside pages of scale 2^55 to 2^63, all keys with like scores: the zeros count in the
    sum of the weights."""
    S, mb = with_scores(i, lambda b, j, k: 0.0 * j)
    page = FORMS[i][4]
    for b, (_, k) in enumerate(S.seqs):
        p = np.arange(-(-k // page))
        zero = (p * page // 384 % 2 == 1) == late
        ids = S.table[b, p]
        S.Vc[ids[zero]] = 0
        S.Ve[ids[zero]] = -64
        S.Ve[ids[~zero]] = S.g.integers(55, 64, (int((~zero).sum()), S.Ve.shape[1]))
    S.upload()
    S.poison()
    S.Q = dev(S.Q, BF)
    check_attention(*attend(B, S, mb, 1.0), S, mb, 1.0)


def test_scales_whose_product_is_no_number_any_more(B):  # noqa: F811
    """Keys under scale 2^-64 times a scale of the scores of 1e-30: all scores are 0, the keys are there all the same."""
    S = Batch8(960, [(3, 300), (70, 200), (1, 9)], 4, 2, 64, 16)
    S.Ke[...] = -64
    S.upload()
    S.poison()
    S.Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), BF)
    A, lse = attend(B, S, 1, 1e-30)
    check_attention(A, lse, S, 1, 1e-30)
    slots = S.table.shape[1] * 16
    score, tags = torch.zeros((3, 2, slots), device="cuda"), torch.zeros((3, 2, slots), dtype=torch.int32, device="cuda")
    B.dllm_paged_weights(S.Q, S.Kp, *S.d, 70, lse, score, slot_pos=tags, K_scale=S.Ks, mask_block=1, scale=1e-30)
    want = np.array([n for n, _ in S.seqs])[:, None] * 2.0
    assert np.abs(score.double().cpu().numpy().sum(-1) - want).max() <= 1e-4 * want.max() and B.check_status() == 0
