"""The fp32 attention's split products hold the outputs to fp32's precision in every instance.

The parity tests bound each element for the worst signs of every rounding, which would let a whole partial
product be lost at 128 dims.  Here the error is taken relative to the outputs' norm, where roundings of either
sign do not add up.  With e = 2^-21 for an operand's two parts and 2^-22 for the low parts' product, which is left out:
* queries and keys are standard normal, so a score's products, each off by 2 e + 2^-22 of itself at most and to either
  side, leave that times sqrt(sum (q_i k_i)^2 / hd) = 1; its sum of hd / 8 steps, cut at 2^-23 each, 16 2^-23 of a
  score of about 1; the exponential 2^-22;
* values are standard normal about 0, so weights that are off by d to either side move the outputs by d of their norm;
* the second product adds 2 e + 2^-22, its sums within and over tiles 24 2^-23.
In all 2 (2 e + 2^-22) + (16 + 2 + 24) 2^-23 = 7.4e-6.  An operand in one TF32 part (2^-12 of itself at most, 10^-4 in
the root mean square) would leave 10^-4."""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth

torch = pytest.importorskip("torch")

TOL = 2 * (2 * 2.0 ** -21 + 2.0 ** -22) + (16 + 2 + 24) * 2.0 ** -23
CASES = [(hd, n_q, new, keys) for hd in (64, 128) for n_q, new, keys in ((2, 3, 1500), (4, 7, 777), (2, 40, 300), (1, 1, 65))]


def split(x):
    """hi + lo as the kernel takes them: 11 bits each, the first rounded, the second cut."""
    x = np.asarray(x, np.float32)
    hi = ((x.view(np.uint32) + np.uint32(0x1000)) & np.uint32(0xffffe000)).view(np.float32)
    lo = ((x - hi).view(np.uint32) & np.uint32(0xffffe000)).view(np.float32)
    return hi.astype(np.float64), lo.astype(np.float64)


def product(a, b, terms):
    """a b^T of split operands with the partial products named in terms, in 64 bits."""
    (ah, al), (bh, bl) = split(a), split(b)
    parts = {"hh": (ah, bh), "hl": (ah, bl), "lh": (al, bh)}
    return sum(parts[t][0] @ parts[t][1].T for t in terms)


def model(q, k, v, s_terms, o_terms):
    s = product(q, k, s_terms) / np.sqrt(q.shape[1])
    w = np.exp(s - s.max(1, keepdims=True)).astype(np.float32)
    return product(w, v.T, o_terms) / w.sum(1, dtype=np.float64, keepdims=True)


@pytest.mark.parametrize("hd,n_q,new,keys", CASES)
def test_the_bound_tells_split_products_from_single_ones(hd, n_q, new, keys):
    """On the formula alone (no GPU): all three partial products are inside the bound, and any one left out is not."""
    g = synth.rng(hd + keys)
    q, k = (g.standard_normal((n, hd), dtype=np.float32) for n in (n_q * new, keys))
    v = g.standard_normal((keys, hd), dtype=np.float32)
    s = q.astype(np.float64) @ k.astype(np.float64).T / np.sqrt(hd)
    w = np.exp(s - s.max(1, keepdims=True))
    ref = w @ v / w.sum(1, keepdims=True)
    err = lambda *t: np.linalg.norm(model(q, k, v, *t) - ref) / np.linalg.norm(ref)   # noqa: E731
    full = ("hh", "hl", "lh")
    assert err(full, full) <= TOL
    for lost in ("hl", "lh"):
        less = tuple(t for t in full if t != lost)
        assert err(less, full) > 5 * TOL and err(full, less) > 5 * TOL


@pytest.mark.gpu
@pytest.mark.parametrize("hd,n_q,new,keys", CASES)
def test_f32_attention_is_as_near_as_its_split_products(hd, n_q, new, keys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_cache_rank_gb300 import binding as B
    from test_gpu_paged import F32, Batch, dev, host
    S = Batch(60 + hd + keys, [(new, keys), (new, 2 * keys + 1)], n_q, 1, hd, 32, F32)
    Q = dev(S.g.standard_normal((S.T, n_q, hd), dtype=np.float32), F32)
    A = host(B.dllm_paged_attention(Q, S.Kp, S.Vp, *S.d, new))
    A0 = paged.attention(host(Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len)[0]
    assert np.linalg.norm(A - A0) <= TOL * np.linalg.norm(A0)
    assert B.check_status() == 0
