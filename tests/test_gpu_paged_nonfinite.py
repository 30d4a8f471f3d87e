"""Attention over a paged cache with queries that are not finite: the formula gives NaN for such a
row and what it gives without it for the others; zeros and -inf stay the mark of a row that sees no key.

The other rows: bit for bit in fp32.  In bf16 a row's maximum may move the reference of the rows in its warp, which
rounds their weights elsewhere, so they are held to the definition with the tolerance of the parity tests."""
import numpy as np
import pytest

from oracle import paged
from test_gpu_paged import B, BF, F32, Batch, check_attention, dev, host  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# seqs (new, keys), n_q, n_kv, hd, mask_block: instances for few rows, one tile and two tiles of rows, each with units
# that one slice holds and units that are cut
CASES = [
    ([(2, 40), (1, 30), (2, 90)], 4, 2, 64, 1),
    ([(2, 9000), (1, 7), (4, 20000)], 4, 2, 128, 1),
    ([(30, 60), (17, 200)], 6, 2, 128, 32),
    ([(33, 20000), (20, 333)], 6, 2, 64, 0),
    ([(300, 300), (150, 700)], 4, 4, 128, 1),
    ([(300, 9000), (200, 203)], 2, 1, 64, 1),
    ([(4, 50), (16, 30000)], 16, 1, 64, 0),
]


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_rows_that_are_not_finite_give_nan(B, i, dt):  # noqa: F811
    seqs, n_q, n_kv, hd, mb = CASES[i]
    S = Batch(700 + i, seqs, n_q, n_kv, hd, 16, dt, pad=1)
    Q = dev(S.g.standard_normal((S.T, n_q, hd), dtype=np.float32), dt)
    call = lambda q, lse: B.dllm_paged_attention(q, S.Kp, S.Vp, *S.d, max(n for n, _ in seqs), mask_block=mb, lse=lse)  # noqa: E731
    la, lb = torch.zeros((S.T, n_q), device="cuda"), torch.zeros((S.T, n_q), device="cuda")
    want = call(Q, la)
    bad = torch.zeros((S.T, n_q), dtype=torch.bool)
    q = Q.clone()
    for x, v in enumerate((float("nan"), float("inf"), -float("inf"), float("nan"), float("inf"))):
        for b in range(len(seqs)):                       # (first rows of a sequence see the fewest keys)
            n, h = int(S.q_start[b]) + (x * seqs[b][0]) // 5, int(S.g.integers(n_q))
            q[n, h, int(S.g.integers(hd))] = v
            bad[n, h] = True
    q[S.rows:] = float("nan")                            # (rows of no sequence)
    got = call(q, lb)
    torch.cuda.synchronize()
    assert torch.isfinite(want[:S.rows]).all() and torch.isfinite(la[:S.rows]).all()
    clean = np.zeros(S.T, bool)
    clean[:S.rows] = ~bad[:S.rows].any(1).numpy()
    bad, ok = bad[:S.rows].cuda(), ~bad[:S.rows].cuda()
    assert torch.isnan(got[:S.rows][bad]).all() and torch.isnan(lb[:S.rows][bad]).all()
    assert torch.isfinite(got[:S.rows][ok]).all() and torch.isfinite(lb[:S.rows][ok]).all()
    if dt == F32:
        assert torch.equal(got[:S.rows][ok], want[:S.rows][ok]) and torch.equal(lb[:S.rows][ok], la[:S.rows][ok])
    else:
        S.Q = Q
        ref = paged.attention(host(Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, mb)
        check_attention(got, lb, ref, S, dt, live=clean)
    assert B.check_status() == 0


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
def test_one_key_and_none(B, dt, hd):  # noqa: F811
    """A row whose one score is -inf is not a row without a key: NaN for the one, zeros and -inf for the other,
    whose queries may be anything."""
    S = Batch(720, [(1, 1), (2, 1), (1, 0), (3, 20), (1, 40)], 2, 1, hd, 8, dt)
    table = S.table.copy()
    table[3, :] = -1                                     # all pages absent
    table[4, 1:] = S.P                                   # the first page alone
    S.d[0].copy_(torch.from_numpy(table))
    S.Kp[:] = 1.0
    Q = torch.full((S.T, 2, hd), 1.0, dtype=dt, device="cuda")
    Q[:, 0, 3] = -float("inf")                           # every score of head 0: -inf
    Q[:, 1, 3] = float("nan")
    for mb in (0, 1):
        lse = torch.zeros((S.T, 2), device="cuda")
        A = B.dllm_paged_attention(Q, S.Kp, S.Vp, *S.d, 3, mask_block=mb, lse=lse)
        torch.cuda.synchronize()
        # rows: (1 key), (before position 0: none with mb 1), (1 key), (no key), 3 x (no page), (8 keys)
        sees = torch.tensor([1, mb == 0, 1, 0, 0, 0, 0, 1], dtype=torch.bool, device="cuda")
        assert torch.isnan(A[sees]).all() and torch.isnan(lse[sees]).all()
        assert not A[~sees].any() and torch.isneginf(lse[~sees]).all()
    assert B.check_status() == 0
