"""Key weights where keys hold infinities or no numbers: their own sums may be anything, all others are what they are without."""
import numpy as np
import pytest

from test_gpu_paged import B, dev  # noqa: F401  (B: the library fixture)
from test_gpu_paged_evict import F8, IDS, KINDS, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("new", [1, 5, 40, 200])
def test_a_key_that_is_no_number_keeps_to_itself(B, kind, new):  # noqa: F811
    """In every form (rows of a tile up to 16, 32, 128, and several tiles), with each new row's lse finite."""
    seqs = [(new, 900), (max(1, new // 2), 333), (new, new)]
    S = make(780 + new, seqs, 6, 2, 64, 16, kind)
    Q = dev(S.g.standard_normal((S.T, 6, 64), dtype=np.float32), S.qdt)
    lse = torch.from_numpy(S.g.random((S.T, 6)).astype(np.float32) + 5).cuda()
    slots = S.table.shape[1] * 16
    before = torch.from_numpy(S.g.random((3, 2, slots)).astype(np.float32)).cuda()

    def run():
        score, tags = before.clone(), torch.zeros((3, 2, slots), dtype=torch.int32, device="cuda")
        B.dllm_paged_weights(Q, S.Kp, *S.d, new, lse, score, slot_pos=tags, K_scale=S.Ks, mask_block=1)
        return score, tags

    want, tags = run()
    bad = torch.zeros((3, 2, slots), dtype=torch.bool, device="cuda")
    raw = S.Kp.view(torch.uint8) if kind == F8 else S.Kp
    values = (0x7f, 0xff) if kind == F8 else (float("nan"), float("inf"), -float("inf"))
    for b, (_, k) in enumerate(seqs):
        for i, j in enumerate(S.g.permutation(k)[:12]):
            h = int(S.g.integers(0, 2))
            raw[int(S.table[b, j // 16]), int(j % 16), h, int(S.g.integers(0, 64))] = values[i % len(values)]
            bad[b, h, j] = True
    got, again = run()
    assert torch.isfinite(want).all() and torch.equal(tags, again)
    assert torch.equal(got[~bad], want[~bad]) and B.check_status() == 0
