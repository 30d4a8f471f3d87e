"""Token sampling where the scaled logits reach the ends of the fp32 range, through the C ABI,
against the fp64 definition.

Tokens are equal and prob is one fp32 rounding of a ratio (2^-24 + 1e-9).  At these magnitudes neighbouring
values are further apart than any filter reaches, so each row has ties of its maximum."""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_cache_rank_gb300 import binding
    binding.lib()
    binding.check_status(reset=True)
    return binding


def check(B, l, u, t=None, k=None, p=None, m=None):
    """Every row is answered (the outputs start as numbers that no answer has) as defined."""
    n, rows = l.shape[:2]
    dev = lambda x, dt=torch.float32: None if x is None else torch.tensor([x] * n, dtype=dt, device="cuda")   # noqa: E731
    out = (torch.full((n, rows), -7, dtype=torch.int32, device="cuda"), torch.full((n, rows), -7.0, device="cuda"))
    B.dllm_sample(l, torch.from_numpy(u).cuda(), temperature=dev(t), top_k=dev(k, torch.int32), top_p=dev(p), min_p=dev(m),
                  out=out)
    tok, prob = (x.cpu().numpy() for x in out)
    lh = l.float().cpu().numpy()
    for b in range(n):
        for i in range(rows):
            rt, rp = paged.sample_row(lh[b, i], u[b, i], 1.0 if t is None else t, k or 0, 1.0 if p is None else p, m or 0.0)
            assert tok[b, i] == rt, (b, i, tok[b, i], rt)
            assert float(prob[b, i]) == pytest.approx(rp, rel=2.0 ** -24 + 1e-9, abs=0.0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [3000, 5000, 40011])
def test_maxima_near_the_largest_number(B, V, dt):
    """Maxima from 1e37 to the type's largest number, alone, tied a few and thousands of times; -max beside them."""
    g = synth.rng(V)
    tops = np.array([1e37, 4.25e37, 4.26e37, 5e37, 1.7e38, torch.finfo(dt).max, -4.26e37, -3e38], np.float32)
    l = -np.abs(g.standard_normal((len(tops), 3, V), dtype=np.float32)) * np.float32(1e38) - np.float32(3.05e38) * (tops < 0)[:, None, None]
    l = np.maximum(l, np.float32(torch.finfo(dt).min))
    for i, top in enumerate(tops):
        for r, ties in enumerate((1, 40, V // 2)):
            l[i, r, g.choice(V, ties, replace=False)] = top
    lt = torch.from_numpy(l).to(dt).cuda()
    assert torch.isfinite(lt).all()
    u = g.random(l.shape[:2]).astype(np.float32)
    for kw in (dict(m=0.1), dict(m=1.0), dict(m=1e-20), dict(m=0.05, p=0.9), dict(p=0.9), dict(k=30), dict(k=30, m=0.1), {},
               dict(t=0.0)):
        check(B, lt, u, **kw)
    assert B.check_status() == 0


@pytest.mark.parametrize("V", [3000, 9001])
def test_the_smallest_normal_temperature(B, V):
    """T = 2^-126: ordinary logits are scaled by 2^126, which is finite, so the row is not greedy."""
    g = synth.rng(V + 5)
    l = np.minimum(g.standard_normal((2, 4, V), dtype=np.float32), np.float32(2.5)).round(2)
    l[:, :, 17] = 2.5
    l[0, 1, 5::7] = 2.5
    lt = torch.from_numpy(l).cuda()
    u = g.random((2, 4)).astype(np.float32)
    for kw in (dict(m=0.1), dict(m=0.1, p=0.9), dict(p=0.9), dict(k=5), {}):
        check(B, lt, u, t=2.0 ** -126, **kw)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [3000, 4100, 9001, 40011])
def test_more_infinite_logits_than_a_chunk_lists(B, V, dt):
    """Rows of 1, 129, 1024, 1025, half and all of V infinite logits, given and by overflow: they share the mass."""
    g = synth.rng(V + 9)
    counts = [c for c in (1, 129, 1024, 1025, V // 2, V) if c <= V]
    l = g.standard_normal((2, len(counts), V), dtype=np.float32)
    for i, c in enumerate(counts):
        l[0, i, g.choice(V, c, replace=False)] = np.inf
        l[1, i, g.choice(V, c, replace=False)] = np.float32(3e38)     # (T = 1/2: past the fp32 range)
    lt = torch.from_numpy(l).to(dt).cuda()
    u = g.random(l.shape[:2]).astype(np.float32)
    # (0.37 and 0.371 of equal weights: no border of the mass falls on a token's edge)
    for kw in (dict(m=0.02), dict(p=0.37), dict(k=30), dict(k=2000), dict(k=900, p=0.371), dict(p=0.37, m=0.5), {}):
        check(B, lt, u, t=0.5, **kw)
    assert B.check_status() == 0
