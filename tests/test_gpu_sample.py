"""GPU parity of the token sampling with its fp64 definition through the C ABI.

Tokens are equal: the kernel sums masses exactly from weights that are within 2^-38 of the
exponential, so a border of the cumulative distribution moves by about 1e-12 of the total and a
test's few thousand uniform numbers, each with some 10^5 borders, meet one with probability
below 1e-3 in all (the seeds are fixed).  prob is one fp32 rounding of a ratio: 2^-24 + 1e-9."""
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


def check(B, logits, u, t=None, k=None, p=None, m=None, valid=None):
    """logits [B, M, V] tensor on the GPU; settings per sequence as lists."""
    f = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda")   # noqa: E731
    kt = None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda")
    vt = None if valid is None else torch.from_numpy(valid).cuda()
    tok, prob = B.dllm_sample(logits, torch.from_numpy(u).cuda(), temperature=f(t), top_k=kt, top_p=f(p), min_p=f(m),
                              valid=vt)
    tok, prob = tok.cpu().numpy(), prob.cpu().numpy()
    l = logits.float().cpu().numpy()
    for b in range(l.shape[0]):
        for i in range(l.shape[1]):
            if valid is not None and not valid[b, i]:
                assert tok[b, i] == -1 and prob[b, i] == 0.0
                continue
            rt, rp = paged.sample_row(l[b, i], u[b, i], 1.0 if t is None else t[b], 0 if k is None else k[b],
                                      1.0 if p is None else p[b], 0.0 if m is None else m[b])
            assert tok[b, i] == rt, (b, i, tok[b, i], rt)
            assert float(prob[b, i]) == pytest.approx(rp, rel=2.0 ** -24 + 1e-9, abs=0.0)
    return tok, prob


@pytest.mark.parametrize("V", [1, 2, 31, 33, 513, 4096, 16384, 16385, 40001, 126464, 152064, 262144])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_filters_at_every_size(B, V, dt):
    g = synth.rng(V)
    Bn, M = 6, 3 if V < 50000 else 1
    l = torch.from_numpy((g.standard_normal((Bn, M, V), dtype=np.float32) * 3)).to(dt).cuda()
    u = g.random((Bn, M)).astype(np.float32)
    t = [1.0, 0.7, 1.3, 0.0, 0.5, 1.0]
    check(B, l, u)
    check(B, l, u, t=t)
    check(B, l, u, t=t, k=[0, 1, 50, 3, V, V - 1])
    check(B, l, u, t=t, p=[0.9, 0.5, 0.999, 0.1, 1.0, 0.0])
    check(B, l, u, t=t, m=[0.0, 0.05, 0.001, 0.5, 1.0, 2.0])
    check(B, l, u, t=t, k=[0, 20, 1000, 5, 40, 7], p=[0.95, 0.9, 0.8, 0.5, 1.0, 0.99], m=[0.02, 0.0, 0.1, 0.3, 0.01, 0.0])


@pytest.mark.parametrize("V", [1000, 40001])
def test_ties_go_to_the_lowest_id(B, V):
    """Rows of few distinct values (bf16 grids, constant rows): cuts fall inside equal values."""
    g = synth.rng(V + 1)
    l = g.integers(0, 4, (5, 4, V)).astype(np.float32)
    l[0] = 1.5
    l[1] = -0.0
    l[1, :, ::2] = 0.0                       # -0 and 0 are one value
    lt = torch.from_numpy(l).cuda()
    u = g.random((5, 4)).astype(np.float32)
    u[:, 0], u[:, 1] = 0.0, np.float32(1.0) - np.float32(2.0 ** -24)
    check(B, lt, u)
    check(B, lt, u, k=[V // 2, 17, 300, 999, 1])
    # (0.37 of equal weights: no border of the mass falls on a token's edge)
    check(B, lt, u, p=[0.37] * 5)
    check(B, lt, u, k=[333] * 5, p=[0.371] * 5)
    check(B, lt, u, t=[0.0] * 5)


def test_masked_infinite_and_nan_logits(B):
    g = synth.rng(9)
    V = 3000
    l = (g.standard_normal((1, 9, V), dtype=np.float32) * 3)
    l[0, 0, 10:] = -np.inf                   # ten left
    l[0, 1] = -np.inf                        # none left
    l[0, 2, ::2] = np.nan
    l[0, 3] = np.nan
    l[0, 4, [5, 77]] = np.inf
    l[0, 5, :] = np.finfo(np.float32).min    # a mask of the type's lowest value everywhere: one value
    l[0, 6, 100:] = np.finfo(np.float32).min
    l[0, 7, 7] = 80.0                        # all mass on one token
    l[0, 8] *= 1e-6                          # nearly flat
    u = np.linspace(0.05, 0.95, 9, dtype=np.float32)[None]
    lt = torch.from_numpy(l).cuda()
    for kw in ({}, dict(k=[20]), dict(p=[0.9]), dict(m=[0.1]), dict(k=[7], p=[0.8], m=[0.01]), dict(t=[0.0])):
        tok, _ = check(B, lt, u, **kw)
        assert tok[0, 1] == -1 and tok[0, 3] == -1 and tok[0, 0] < 10 and tok[0, 2] % 2 == 1
        assert tok[0, 4] in (5, 77) and tok[0, 6] < 100 and tok[0, 7] == 7
    valid = np.array([[1, 0, 1, 0, 1, 1, 0, 1, 1]], np.uint8)
    check(B, lt, u, k=[20], valid=valid)


def test_wide_kept_sets_and_extreme_scales(B):
    """Nearly flat rows keep tens of thousands of tokens (more than a CTA lists); logits far
    from 0, where an fp32 step is wider than the differences that matter, and temperatures that
    stretch them."""
    g = synth.rng(77)
    V = 60011
    l = (g.standard_normal((6, 2, V), dtype=np.float32) * np.array([0.01, 1.0, 0.3, 2.0, 5.0, 1.0], np.float32)[:, None, None])
    l[3] += 3.0e5
    l[4] -= 2.0e7
    l[5] *= 3.0e8
    lt = torch.from_numpy(l.astype(np.float32)).cuda()
    u = g.random((6, 2)).astype(np.float32)
    check(B, lt, u)
    check(B, lt, u, p=[0.9, 0.99, 0.5, 0.9, 0.9, 0.9])
    check(B, lt, u, k=[20000, 30000, 59999, 100, 5, 3], p=[0.9, 1.0, 0.97, 1.0, 0.9, 0.5])
    check(B, lt, u, m=[0.9, 0.01, 0.3, 0.1, 0.1, 0.1], t=[1.0, 2.0, 0.05, 50.0, 1000.0, 1e7])
    check(B, lt.bfloat16(), u, p=[0.9] * 6, t=[1.0, 1.0, 0.5, 9.0, 3.0, 1e8])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_flat_rows_of_a_large_vocabulary(B, dt):
    """Prefixes of 10^4 to 1.5 10^5 tokens under top-p alone, with the chunks' shares uneven, and under
    min-p beside it."""
    g = synth.rng(80)
    V = 150001
    l = g.standard_normal((8, 2, V), dtype=np.float32) * np.array([0.3, 1, 1, 1.5, 2, 2.5, 3, 3.5], np.float32)[:, None, None]
    l[2, 1, :40000] += 1.0
    l[4, 0, 70000:] -= 6.0
    l[5, 1, 100:] = -np.inf
    l[6, 0, ::3] = np.nan
    lt = torch.from_numpy(l).to(dt).cuda()
    u = g.random((8, 2)).astype(np.float32)
    check(B, lt, u, p=[0.5, 0.9, 0.95, 0.9, 0.97, 0.99, 0.999, 0.97])
    check(B, lt, u, p=[0.9999, 0.99, 0.1, 0.999, 0.95, 0.9, 0.99, 0.99], t=[1.0, 0.9, 1.3, 1.0, 0.8, 1.2, 1.5, 0.9])
    check(B, lt, u, p=[0.99] * 8, m=[0.3, 0.01, 0.001, 0.0, 0.002, 1e-4, 1e-6, 1e-9])
    assert B.check_status() == 0


def test_rows_that_start_anywhere(B):
    """Logits whose base is aligned to their element alone."""
    g = synth.rng(78)
    for dt in (torch.float32, torch.bfloat16):
        for V in (1001, 20003):
            buf = torch.from_numpy(g.standard_normal(2 * 3 * V + 8, dtype=np.float32) * 3).to(dt).cuda()
            for off in (0, 1, 3, 7):
                l = buf[off:off + 6 * V].view(2, 3, V)
                u = g.random((2, 3)).astype(np.float32)
                check(B, l, u)
                check(B, l, u, t=[0.7, 0.0], k=[40, 0], p=[0.9, 0.9])


@pytest.mark.parametrize("V", [900, 30011])
def test_settings_that_are_nan_or_past_their_range(B, V):
    """NaN temperatures are greedy, NaN top_p and min_p off; top_p <= 0 and min_p > 1 leave the maximum,
    negative min_p and top_k are off."""
    g = synth.rng(79)
    l = torch.from_numpy(g.standard_normal((8, 1, V), dtype=np.float32) * 2).cuda()
    u = g.random((8, 1)).astype(np.float32)
    n = float("nan")
    check(B, l, u, t=[n, -1.0, 0.0, -n, 1.0, 1.0, 1.0, 1e-39])
    want, prob = check(B, l, u)
    tok, pr = B.dllm_sample(l, torch.from_numpy(u).cuda(), top_p=torch.full((8,), n, device="cuda"),
                            min_p=torch.full((8,), n, device="cuda"), top_k=torch.full((8,), -4, dtype=torch.int32, device="cuda"))
    assert np.array_equal(tok.cpu().numpy(), want) and np.array_equal(pr.cpu().numpy(), prob)
    for kw in ({"p": [0.0] * 8}, {"p": [-3.0] * 8}, {"m": [1.0] * 8}, {"m": [5.0] * 8}, {"m": [float("inf")] * 8}):
        tok, pr = check(B, l, u, **kw)
        assert np.array_equal(tok[:, 0], l[:, 0].argmax(-1).cpu().numpy()) and (pr == 1.0).all()
    check(B, l, u, m=[-1.0, -0.5, 0.0, -9.0, -1.0, -2.0, -3.0, -4.0], p=[2.0, 9.0] * 4)


def test_uniform_numbers_outside_their_range_take_the_nearer_end(B):
    l = torch.tensor([[[0.0, 1.0, 2.0]] * 6], device="cuda")
    u = torch.tensor([[-1.0, float("nan"), 1.0, 7.0, float("inf"), 0.0]], device="cuda")
    tok, _ = B.dllm_sample(l, u)
    assert tok.tolist() == [[0, 0, 2, 2, 2, 0]]


def test_frequencies_follow_the_distribution(B):
    """20000 rows of one distribution: each token's count within 5 standard deviations."""
    V, n = 12, 20000
    l = torch.arange(V, dtype=torch.float32, device="cuda")[None, None] * 0.3
    g = synth.rng(4)
    u = torch.from_numpy(g.random((1, n)).astype(np.float32)).cuda()
    tok, prob = B.dllm_sample(l.expand(1, n, V).contiguous(), u)
    p = torch.softmax(l[0, 0].double(), -1).cpu().numpy()
    c = np.bincount(tok.cpu().numpy()[0], minlength=V)
    assert (np.abs(c - n * p) <= 5 * np.sqrt(n * p * (1 - p))).all()
    np.testing.assert_allclose(prob.cpu().numpy()[0], p[tok.cpu().numpy()[0]], rtol=1e-6)


def test_repeats_replays_and_writes_inside(B):
    from test_gpu_guards import Guarded
    G = Guarded(21)
    g = synth.rng(22)
    Bn, M, V = 3, 5, 20011
    l = G.new((Bn, M, V), torch.float32, torch.from_numpy(g.standard_normal((Bn, M, V), dtype=np.float32) * 3))
    u = G.new((Bn, M), torch.float32, torch.from_numpy(g.random((Bn, M)).astype(np.float32)))
    t, p = G.new((Bn,), torch.float32, torch.tensor([0.7, 1.0, 0.0])), G.new((Bn,), torch.float32, torch.tensor([0.9] * 3))
    k = G.new((Bn,), torch.int32, torch.tensor([0, 30, 9], dtype=torch.int32))
    out = (G.new((Bn, M), torch.int32), G.new((Bn, M), torch.float32))
    B.dllm_sample(l, u, t, k, p, out=out)
    first = [x.clone() for x in out]
    ws = G.new((int(B.lib().dllm_sample_workspace_bytes(Bn, M, V)),), torch.uint8)
    B.dllm_sample(l, u, t, k, p, out=out, ws=ws)
    assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    for _ in range(3):
        B.dllm_sample(l, u, t, k, p, out=out)
        assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        B.dllm_sample(l, u, t, k, p, out=out)
    l.mul_(0.5)
    gr.replay()
    torch.cuda.synchronize()
    for b in range(Bn):
        for i in range(M):
            rt, _ = paged.sample_row(l[b, i].cpu().numpy(), float(u[b, i]), float(t[b]), int(k[b]), float(p[b]))
            assert int(out[0][b, i]) == rt
    assert B.check_status() == 0
    G.check()
