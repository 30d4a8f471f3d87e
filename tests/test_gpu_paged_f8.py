"""GPU parity of the 8-bit pages with their fp64 definitions: codes and scales that new rows leave, attention over
them, at ragged lengths, odd sizes, masks that leave rows empty, absent pages, far positions, scales far apart.

Tolerances (u = half a step, relative: bf16 2^-8, fp16 2^-11, E4M3 2^-4):
* append: a value carries 2e-6 of its pair's length (test_gpu_paged.py), then one rounding to E4M3: u |x|, or half of
  the subnormal step, 2^-10.  An exponent may differ by one where the rows' maximum is that near 448 2^e.
* attention: a query's two parts miss 2^-17 of its largest element in every dim (half of the subnormal step, 2^-10, where
  the largest is 2^7 or more), fp32 sums hd 2^-23 |q| |k| (both
  times the scale: ds); a weight exp(+-2 ds), 1e-5 for the exponential, u(fp16), and u(E4M3)^2 = 2^-8 for its two
  parts, or 2^-17 of the row's largest weight times value scale (oracle.paged.weight_floor); the output u |A|.
"""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth
from test_gpu_paged import ATTEND, BF, F32, B, dev, host  # noqa: F401  (B: the library fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Batch8:
    """Sequences of (new rows, keys) over a shuffled pool of 8-bit pages; what is no key is NaN."""

    def __init__(self, seed, seqs, n_q, n_kv, hd, page, pad=0, spare=3, max_pages=None, spread=0, scale=1.0):
        self.g = g = synth.rng(seed)
        self.seqs, self.n_q, self.n_kv, self.hd, self.page = seqs, n_q, n_kv, hd, page
        need = [-(-k // page) for _, k in seqs]
        self.P = sum(need) + spare
        ids = g.permutation(self.P).astype(np.int32)
        self.table = np.full((len(seqs), max_pages or max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            m = min(n, self.table.shape[1])
            self.table[b, :m] = ids[at:at + m]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.kv_len = np.array([k for _, k in seqs], np.int32)
        self.rows = int(self.q_start[-1])
        self.T = self.rows + pad
        shape = (self.P, page, n_kv, hd)
        # codes of a normal distribution of 100, the scales 2^-7 times a power of two within +-spread
        self.Kc = paged.e4m3(g.standard_normal(shape) * 100)
        self.Vc = paged.e4m3(g.standard_normal(shape) * 100)
        self.Ke = -7 + g.integers(-min(spread, 2), min(spread, 2) + 1, (self.P, n_kv)) + int(np.log2(scale))
        self.Ve = -7 + g.integers(-spread, spread + 1, (self.P, n_kv))
        self.d = [torch.from_numpy(a).cuda() for a in (self.table, self.q_start, self.kv_len)]
        self.upload()

    def upload(self):
        self.Kp, self.Vp = (torch.from_numpy(c).float().cuda().to(E4M3) for c in (self.Kc, self.Vc))
        self.Ks, self.Vs = (torch.from_numpy((e + 127).astype(np.uint8)).cuda().view(E8M0) for e in (self.Ke, self.Ve))

    def used(self):
        used = np.zeros((self.P, self.page), bool)
        for b, (_, k) in enumerate(self.seqs):
            for j in range(min(k, self.table.shape[1] * self.page)):
                p = self.table[b, j // self.page]
                if 0 <= p < self.P:
                    used[p, j % self.page] = True
        return used

    def poison(self):
        """NaN codes in every slot that no sequence has a key in, and 0xff in the scales of pages without one."""
        used = self.used()
        m = torch.from_numpy(~used).cuda()
        for t in (self.Kp, self.Vp):
            t.view(torch.uint8)[m] = 0x7f
        for t in (self.Ks, self.Vs):
            t.view(torch.uint8)[torch.from_numpy(~used.any(1)).cuda()] = 0xff

    def values(self):
        return self.Kc * 2.0 ** self.Ke[:, None, :, None], self.Vc * 2.0 ** self.Ve[:, None, :, None]

    def cache(self):
        return (self.Kp, self.Vp, self.Ks, self.Vs, *self.d)


def exps(t):
    return t.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


# ---------------------------------------------------------------------------- append
APPEND = [
    # seqs (new, keys), n_q, n_kv, hd, page, in, norm, rope, pad, base
    ([(1, 1)], 1, 1, 64, 8, F32, True, True, 0, False),
    ([(32, 1024)], 32, 32, 128, 64, BF, False, True, 0, False),
    ([(1, 77), (1, 16), (0, 5), (1, 3000), (1, 1)], 28, 4, 128, 16, F32, True, True, 5, True),
    ([(67, 130), (0, 0), (5, 5), (33, 4097)], 12, 4, 64, 32, BF, True, True, 9, False),
    ([(40, 100007), (3, 131072)], 8, 1, 128, 256, F32, True, True, 1, True),     # far positions
    ([(19, 19), (7, 40)], 5, 5, 64, 128, F32, False, False, 0, False),
    ([(700, 900), (3, 1030)], 2, 1, 128, 256, BF, False, True, 0, False),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
@pytest.mark.parametrize("loud", [0, 6])
def test_append_parity(B, i, loud):  # noqa: F811
    """loud: rows 2^6 times as large as the codes in the pages, so that scales grow and earlier rows are rounded anew."""
    seqs, n_q, n_kv, hd, page, dti, norm, rope, pad, based = APPEND[i]
    S = Batch8(100 + i, seqs, n_q, n_kv, hd, page, pad)
    qkv = dev(S.g.standard_normal((S.T, n_q + 2 * n_kv, hd), dtype=np.float32) * 2.0 ** loud, dti)
    Q, K, V = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    gq = dev(1 + 0.1 * S.g.standard_normal(hd), BF) if norm else None
    gk = dev((1 + 0.1 * S.g.standard_normal(hd)) * 2.0 ** loud, BF) if norm else None
    f = (10000.0 ** (-2 * np.arange(hd // 2) / hd)).astype(np.float32) if rope else None
    base = S.g.integers(-3, 5000, len(seqs)).astype(np.int32) if based else None
    Qo = torch.full((S.T, n_q, hd), 7.0, dtype=BF, device="cuda")
    before = {n: t.view(torch.uint8).clone() for n, t in (("K", S.Kp), ("V", S.Vp))}
    out = B.dllm_paged_append_f8(K, V, *S.cache(), Q=Q, Q_out=Qo, gamma_q=gq, gamma_k=gk, eps=1e-6,
                                 inv_freq=None if f is None else torch.from_numpy(f).cuda(),
                                 pos_base=None if base is None else torch.from_numpy(base).cuda())
    assert out is Qo
    h = {n: None if t is None else host(t) for n, t in (("q", gq), ("k", gk))}
    ref, Qr, lost = paged.append_f8(host(K), host(V), S.Kc, S.Vc, S.Ke, S.Ve, S.table, S.q_start, S.kv_len, Q=host(Q),
                                    Q_out=np.full((S.T, n_q, hd), 7.0), gamma_q=h["q"], gamma_k=h["k"], eps=1e-6,
                                    inv_freq=f, pos_base=base)
    assert lost == 0 and B.check_status() == 0
    assert (Qo[S.rows:] == 7.0).all()
    pair = np.hypot(Qr[..., :hd // 2], Qr[..., hd // 2:])
    tol = 2.0 ** -8 * np.abs(Qr) + 2e-6 * np.concatenate([pair, pair], -1)
    assert (np.abs(host(Qo) - Qr) <= tol).all()
    for n, codes, scale in (("K", S.Kp, S.Ks), ("V", S.Vp, S.Vs)):
        c0, e0, wrote = ref[n]
        e = exps(scale)
        assert np.array_equal(e, e0)          # (no maximum of these inputs is within 1e-6 of 448 2^e)
        same = torch.from_numpy(~wrote).cuda()
        assert torch.equal(codes.view(torch.uint8)[same], before[n][same])    # other slots: bit for bit
        got, want = host(codes)[wrote], c0[wrote]
        p = np.hypot(want[..., :hd // 2], want[..., hd // 2:]) if n == "K" else np.zeros(want.shape[:-1] + (hd // 2,))
        tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 4e-6 * np.concatenate([p, p], -1)
        assert (np.abs(got - want) <= tol).all()
        if n == "V":                           # no arithmetic before the rounding: the codes themselves
            assert np.array_equal(got, paged.e4m3(want))


def test_append_zeros_extremes_and_nan(B):  # noqa: F811
    """A page of zeros takes the least scale; magnitudes past 448 2^63 saturate; a NaN stays one and leaves
    the scale to the other rows; values at a border of the scale fall on its side."""
    S = Batch8(5, [(6, 6)], 1, 1, 64, 8)
    x = torch.zeros((6, 1, 64), device="cuda")
    V = x.clone()
    V[0, 0, 0], V[1, 0, 1], V[2, 0, 2] = 3e38, -float("inf"), float("nan")
    B.dllm_paged_append_f8(x, V, *S.cache())
    p = S.table[0, 0]
    assert exps(S.Ks)[p, 0] == -64 and not host(S.Kp)[p, :6].any()
    v = host(S.Vp)[p, :6, 0]
    assert exps(S.Vs)[p, 0] == 63 and v[0, 0] == 448 and v[1, 1] == -448 and np.isnan(v[2, 2])
    assert np.count_nonzero(np.nan_to_num(v, nan=1.0)) == 3
    for top, e in ((448.0, 0), (np.nextafter(np.float32(448), np.float32(500)), 1), (1.75, -8), (1e-30, -64), (2.0 ** 70, 62)):
        x.fill_(0.0)
        x[3, 0, 5] = float(top)
        B.dllm_paged_append_f8(x, x, *S.cache())
        assert exps(S.Ks)[p, 0] == e == paged.exponent_for(float(np.float32(top)))


def test_append_rows_without_a_page_and_keys_alone(B):  # noqa: F811
    S = Batch8(8, [(10, 20), (4, 40), (5, 3)], 1, 1, 64, 8, max_pages=4)
    table = S.table.copy()
    table[0, 1] = S.P                                  # outside the pool: positions 10 .. 15 lost
    S.table, S.d[0] = table, torch.from_numpy(table).cuda()     # sequence 1: positions 36 .. 39 past the table
    K, V, Q = (dev(S.g.standard_normal((S.T, 1, 64), dtype=np.float32), F32) for _ in range(3))
    Qo = torch.full((S.T, 1, 64), 3.0, dtype=BF, device="cuda")
    kb = S.Kp.view(torch.uint8).clone()
    B.dllm_paged_append_f8(K, V, *S.cache(), Q=Q, Q_out=Qo)
    ref, Qr, lost = paged.append_f8(host(K), host(V), S.Kc, S.Vc, S.Ke, S.Ve, table, S.q_start, S.kv_len, Q=host(Q),
                                    Q_out=np.full((S.T, 1, 64), 3.0))
    assert lost == 10 and B.check_status(reset=True) == B.STATUS_PAGE
    c0, e0, wrote = ref["K"]
    assert np.array_equal(exps(S.Ks), e0) and np.array_equal(host(S.Kp)[wrote], paged.e4m3(c0[wrote]))
    assert torch.equal(S.Kp.view(torch.uint8)[torch.from_numpy(~wrote).cuda()], kb[torch.from_numpy(~wrote).cuda()])
    assert torch.equal(Qo.cpu(), torch.from_numpy(Qr).float().to(BF))
    assert B.dllm_paged_append_f8(K, V, *S.cache()) is None
    B.check_status(reset=True)


# ---------------------------------------------------------------------------- attention
def check_attention(got, lse, S, mb, scale=None, live=None):
    Kv, Vv = S.values()
    A, Aa, L, n = paged.attention(host(S.Q), Kv, Vv, S.table, S.q_start, S.kv_len, mb, scale)
    Fl = paged.weight_floor(host(S.Q), Kv, S.Vc, S.Ve, S.table, S.q_start, S.kv_len, mb, scale)
    live = np.arange(S.T) < S.rows if live is None else live
    used = S.used()
    kn = np.linalg.norm(Kv, axis=-1)[used].max() if used.any() else 0.0
    k1 = np.abs(Kv).sum(-1)[used].max() if used.any() else 0.0
    Q = host(S.Q)
    ds = (S.hd * 2.0 ** -23 * np.linalg.norm(Q, axis=-1) * kn + 2.0 ** -17 * np.abs(Q).max(-1) * k1) * (scale or S.hd ** -0.5)
    rel = 2 * ds[..., None] + n[:, None, None] * 2.0 ** -23 + 1e-5
    tol = 2.0 ** -8 * np.abs(A) + Aa * (rel + 2.0 ** -11 + 2.0 ** -8) * 1.01 + 2.0 ** -17 * Fl * 1.01 + 1e-30
    err = np.abs(host(got) - A)
    assert np.isfinite(host(got)[live]).all()
    assert (err[live] <= tol[live]).all(), (err - tol)[live].max()
    if lse is not None:
        l = host(lse)[live]
        assert np.array_equal(np.isneginf(l), np.isneginf(L[live]))
        ok = np.isfinite(L[live])
        lt = (ds + n[:, None] * 2.0 ** -23 + 1e-5 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0)))[live]
        assert (np.abs(l[ok] - L[live][ok]) <= lt[ok]).all(), np.abs(l[ok] - L[live][ok]).max()
    return A


# forms: the rows of a key head in a unit (up to 8, 16, 32, 64, and 128 shared by two streams)
FORMS = ATTEND + [
    ([(2, 333), (1, 1000)], 12, 3, 128, 8, 1, 0),
    ([(4, 500), (3, 70)], 16, 4, 64, 16, 0, 2),
    ([(32, 2000), (31, 32)], 2, 2, 128, 64, 0, 0),
    ([(60, 1500), (10, 200)], 3, 3, 128, 32, 1, 0),
    ([(21, 800)], 3, 1, 64, 128, 16, 0),
    ([(1, 20000)], 8, 8, 128, 64, 0, 0),
]


def attend_case(B, i, spread):  # noqa: F811
    seqs, n_q, n_kv, hd, page, mb, pad = FORMS[i]
    S = Batch8(300 + i, seqs, n_q, n_kv, hd, page, pad, spread=spread)
    S.poison()
    S.Q = dev(S.g.standard_normal((S.T, n_q, hd), dtype=np.float32) * 1.5, BF)
    A = torch.full((S.T, n_q, hd), 5.0, dtype=BF, device="cuda")
    lse = torch.full((S.T, n_q), 5.0, device="cuda")
    out = B.dllm_paged_attention_f8(S.Q, *S.cache(), max(n for n, _ in seqs), mask_block=mb, A=A, lse=lse)
    assert out is A and B.check_status() == 0
    assert (A[S.rows:] == 5.0).all() and (lse[S.rows:] == 5.0).all()      # padded rows: as they were
    check_attention(A, lse, S, mb)
    return S, A


@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_attention_parity(B, i, spread):  # noqa: F811
    """spread: page scales up to 2^6 apart either way (values; keys 2^2)."""
    attend_case(B, i, spread)


def test_attention_absent_pages_and_short_tables(B):  # noqa: F811
    """Entries outside the pool and keys past the table are absent; a row with none gets zeros."""
    S = Batch8(40, [(3, 90), (2, 40), (35, 300), (1, 10)], 4, 2, 64, 16, max_pages=10)
    S.table[0, 1], S.table[0, 3] = -1, S.P
    S.table[1, :] = -5
    S.table[2, :9] = 1 << 30
    S.d[0] = torch.from_numpy(S.table).cuda()
    S.poison()
    S.Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), BF)
    for mb in (0, 1):
        lse = torch.empty((S.T, 4), device="cuda")
        A = B.dllm_paged_attention_f8(S.Q, *S.cache(), 35, mask_block=mb, lse=lse)
        ref = check_attention(A, lse, S, mb)
        assert (ref == 0).all((1, 2)).any() and not host(A)[(ref == 0).all((1, 2))].any()
    assert B.check_status() == 0


@pytest.mark.parametrize("n_q", [2, 16, 60, 200])
def test_attention_climbing_maxima_and_value_scales(B, n_q):  # noqa: F811
    """Scores that grow along the keys by far more than an exponent's range, then fall, while the values'
    scales rise against them: references move in both, at every form, with strided queries."""
    n, hd = 1500, 64
    S = Batch8(41 + n_q, [(2, n), (1, n)], n_q, 2, hd, 32)
    ramp = np.concatenate([np.linspace(-40, 40, 900), np.linspace(40, -60, 600)])
    S.Kc[...] = 0
    S.Ke[...] = -3
    S.Ve[...] = -20
    for b in range(2):
        for j in range(n):
            S.Kc[S.table[b, j // 32], j % 32, :, 0] = paged.e4m3(ramp[j] * 8)
            S.Ve[S.table[b, j // 32]] = -20 + 40 * j // n
    S.upload()
    wide = dev(S.g.standard_normal((S.T, n_q + 3, hd), dtype=np.float32), BF)
    wide[:, 1:1 + n_q, 0] = 30.0
    wide[:, 1:1 + n_q:2, 0] = 2.0
    S.Q = wide[:, 1:1 + n_q]
    lse = torch.empty((S.T, n_q), device="cuda")
    A = B.dllm_paged_attention_f8(S.Q, *S.cache(), 2, mask_block=0, scale=0.25, lse=lse)
    check_attention(A, lse, S, 0, 0.25)


def test_attention_queries_of_all_sizes_and_not_finite(B):  # noqa: F811
    """Queries from 1e-30 to 1e30 of their own row's scale, zeros, NaN and infinities: each row to itself."""
    S = Batch8(55, [(9, 400), (1, 130)], 4, 2, 128, 16)
    q = S.g.standard_normal((S.T, 4, 128)).astype(np.float32)
    q[0] *= 1e-30
    q[1] *= 1e-3
    q[2] = 0
    q[3, :, 5:] *= 2.0 ** -12                     # one loud element
    S.Q = dev(q, BF)
    lse = torch.empty((S.T, 4), device="cuda")
    A = B.dllm_paged_attention_f8(S.Q, *S.cache(), 9, mask_block=1, lse=lse)
    check_attention(A, lse, S, 1)
    bad = S.Q.clone()
    bad[4, 1, 7], bad[5, 0, 0], bad[6, 3, 3] = float("nan"), float("inf"), -float("inf")
    got = B.dllm_paged_attention_f8(bad, *S.cache(), 9, mask_block=1)
    hit = torch.zeros((S.T, 4), dtype=torch.bool, device="cuda")
    hit[4, 1] = hit[5, 0] = hit[6, 3] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], A[~hit])


def test_attention_repeats_bit_for_bit_and_replays_new_lengths(B):  # noqa: F811
    S, A = attend_case(B, 4, 2)
    for _ in range(3):
        assert torch.equal(B.dllm_paged_attention_f8(S.Q, *S.cache(), 67, mask_block=1)[:S.rows], A[:S.rows])
    out = torch.zeros_like(A)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.dllm_paged_attention_f8(S.Q, *S.cache(), 67, mask_block=1, A=out)
    B.dllm_paged_attention_f8(S.Q, *S.cache(), 67, mask_block=0)      # (other work in between)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:S.rows], A[:S.rows])
    kv, starts = S.kv_len.copy(), S.q_start.copy()
    kv[3] -= 1000
    kv[2] = 2
    starts[1:4] -= 30                       # 37 rows in the first sequence, 63 in the fourth
    S.kv_len, S.q_start = kv, starts
    S.d[1].copy_(torch.from_numpy(starts))
    S.d[2].copy_(torch.from_numpy(kv))
    g.replay()
    torch.cuda.synchronize()
    check_attention(out, None, S, 1)


def test_rows_outside_the_bounds_are_left_alone(B):  # noqa: F811
    S = Batch8(42, [(50, 400), (3, 90), (20, 700)], 4, 2, 64, 16)
    S.Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), BF)
    for most in (1, 3, 7, 15, 33, 49):
        A = torch.full((S.T, 4, 64), 9.0, dtype=BF, device="cuda")
        B.dllm_paged_attention_f8(S.Q, *S.cache(), most, mask_block=1, A=A)
        slot = np.concatenate([np.arange(n) for n, _ in S.seqs])
        inside = torch.from_numpy(slot < most).cuda()
        assert (A[~inside] == 9.0).all() and not (A[inside] == 9.0).all(-1).any()
        check_attention(A, None, S, 1, live=slot < most)
    # the last sequence's rows reach past T; the one before has descending starts
    T, d1 = 60, torch.tensor([0, 50, 40, 80], dtype=torch.int32, device="cuda")
    A = torch.full((T, 4, 64), 9.0, dtype=BF, device="cuda")
    B.dllm_paged_attention_f8(S.Q[:T], S.Kp, S.Vp, S.Ks, S.Vs, S.d[0], d1, S.d[2], 50, mask_block=1, A=A)
    assert torch.isfinite(A).all() and (A[50:] != 9.0).any()
    kv = torch.zeros((T, 2, 64), dtype=BF, device="cuda")
    B.dllm_paged_append_f8(kv, kv, S.Kp, S.Vp, S.Ks, S.Vs, S.d[0], d1, S.d[2], Q=S.Q[:T])
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    A = torch.full((5, 4, 64), 9.0, dtype=BF, device="cuda")
    B.dllm_paged_attention_f8(S.Q[:5], S.Kp, S.Vp, S.Ks, S.Vs, S.d[0], zero, S.d[2], 5, A=A)
    assert (A == 9.0).all()
    e = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    assert B.dllm_paged_attention_f8(e, S.Kp, S.Vp, S.Ks, S.Vs, S.d[0], zero, S.d[2], 5).shape == (0, 4, 64)
    assert B.dllm_paged_append_f8(e[:, :2], e[:, :2], S.Kp, S.Vp, S.Ks, S.Vs, S.d[0], zero, S.d[2], Q=e).shape == (0, 4, 64)
    assert B.check_status(reset=True) in (0, B.STATUS_PAGE)


def test_as_many_sequences_as_a_batch_may_have(B):  # noqa: F811
    g = synth.rng(43)
    seqs = [(0 if b % 3 == 1 else 1 + b % 4, 0) for b in range(1024)]
    seqs = [(n, n + (0 if b % 7 == 0 else int(g.integers(0, 150)))) for b, (n, _) in enumerate(seqs)]
    S = Batch8(44, seqs, 6, 2, 64, 8)
    K, V, Q = (dev(S.g.standard_normal((S.T, h, 64), dtype=np.float32), BF) for h in (2, 2, 6))
    S.Q = B.dllm_paged_append_f8(K, V, *S.cache(), Q=Q)
    assert torch.equal(S.Q, Q)
    ref, _, _ = paged.append_f8(host(K), host(V), S.Kc, S.Vc, S.Ke, S.Ve, S.table, S.q_start, S.kv_len)
    S.Kc, S.Vc, S.Ke, S.Ve = paged.e4m3(ref["K"][0]), paged.e4m3(ref["V"][0]), ref["K"][1], ref["V"][1]
    assert np.array_equal(host(S.Kp), S.Kc) and np.array_equal(host(S.Vp), S.Vc)
    assert np.array_equal(exps(S.Ks), S.Ke) and np.array_equal(exps(S.Vs), S.Ve)
    lse = torch.empty((S.T, 6), device="cuda")
    A = B.dllm_paged_attention_f8(S.Q, *S.cache(), 4, mask_block=1, lse=lse)
    check_attention(A, lse, S, 1)
    assert B.check_status() == 0


def test_writes_stay_inside_their_arrays(B):  # noqa: F811
    from test_gpu_guards import Guarded
    seqs = [(33, 100), (1, 4000), (130, 130)]
    S = Batch8(50, seqs, 6, 2, 128, 16, pad=2)
    G = Guarded(51)
    u8 = [G.new(t.shape, torch.uint8, t.view(torch.uint8)) for t in (S.Kp, S.Vp, S.Ks, S.Vs)]
    cache = [u8[0].view(E4M3), u8[1].view(E4M3), u8[2].view(E8M0), u8[3].view(E8M0)]
    d = [G.new(t.shape, torch.int32, t) for t in S.d]
    Q, K, V = (G.new((S.T, h, 128), BF, torch.randn((S.T, h, 128)).to(BF)) for h in (6, 2, 2))
    Qo, A, lse = G.new((S.T, 6, 128), BF), G.new((S.T, 6, 128), BF), G.new((S.T, 6), F32)
    B.dllm_paged_append_f8(K, V, *cache, *d, Q=Q, Q_out=Qo)
    for most in (130, 9, 5, 2, 1):
        ws = G.new((max(16, B.dllm_paged_attention_f8_workspace_bytes(S.T, 3, most, 6, 2, 128)),), torch.uint8)
        for mb in (0, 1):
            B.dllm_paged_attention_f8(Qo, *cache, *d, most, mask_block=mb, A=A, lse=lse, ws=ws)
    assert B.check_status() == 0
    G.check()
