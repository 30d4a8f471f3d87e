"""GPU parity of the paged append and the paged attention with their fp64 definitions, through
the C ABI, at ragged lengths, odd sizes, masks that leave rows empty, absent pages, strided
rows and padded batches; untouched memory stays untouched.

Tolerances (u = half a step of the output type: 2^-8 bf16, 2^-24 fp32):
* append: a rotated element carries the angle's fp32 rounding after reduction (1.2e-7 rad), that of
  sin and cos, and of a handful of fp32 operations, each relative to its pair's length:
  2e-6 * sqrt(x^2 + y^2) in all, then one rounding u * |value|.
* attention: a score's fp32 accumulation errs by hd 2^-23 |q| |k| scale (ds), a weight by the
  factor exp(+-2 ds) and 1e-5 for the exponential, n accumulated terms by n 2^-23 of the sum of
  weight * |v| (A_abs), the output by u |A|; bf16 weights are rounded once more (u A_abs).
"""
import numpy as np
import pytest

from oracle import paged
from sparse_kv_cache_rank_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_cache_rank_gb300 import binding
    binding.lib()
    binding.check_status(reset=True)
    return binding


def dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()


def host(t):
    return t.double().cpu().numpy()


class Batch:
    """Sequences of (new rows, keys) over a shuffled page pool; slots past the keys hold NaN."""

    def __init__(self, seed, seqs, n_q, n_kv, hd, page, dt, pad=0, spare=3, max_pages=None, scale=1.0):
        self.g = g = synth.rng(seed)
        self.seqs, self.n_q, self.n_kv, self.hd, self.page, self.dt = seqs, n_q, n_kv, hd, page, dt
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
        self.Kp = dev(g.standard_normal(shape, dtype=np.float32) * scale, dt)
        self.Vp = dev(g.standard_normal(shape, dtype=np.float32), dt)
        self.d = [torch.from_numpy(a).cuda() for a in (self.table, self.q_start, self.kv_len)]

    def poison(self):
        """NaN in every slot that no sequence has a key in."""
        used = np.zeros((self.P, self.page), bool)
        for b, (_, k) in enumerate(self.seqs):
            for j in range(min(k, self.table.shape[1] * self.page)):
                p = self.table[b, j // self.page]
                if 0 <= p < self.P:
                    used[p, j % self.page] = True
        m = torch.from_numpy(~used).cuda()
        self.Kp[m] = float("nan")
        self.Vp[m] = float("nan")


# ---------------------------------------------------------------------------- append
APPEND = [
    # seqs (new, keys), n_q, n_kv, hd, page, in, cache, norm, rope, pad
    ([(1, 1)], 1, 1, 64, 8, F32, F32, True, True, 0),
    ([(32, 1024)], 32, 32, 128, 64, BF, BF, False, True, 0),
    ([(1, 77), (1, 16), (0, 5), (1, 3000), (1, 1)], 28, 4, 128, 16, F32, BF, True, True, 5),
    ([(67, 130), (0, 0), (5, 5), (33, 4097)], 12, 4, 64, 32, BF, BF, True, True, 9),
    ([(40, 100007), (3, 131072)], 8, 1, 128, 256, F32, F32, True, True, 1),     # far positions
    ([(19, 19), (7, 40)], 5, 5, 64, 128, F32, F32, False, False, 0),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append_parity(B, i):
    seqs, n_q, n_kv, hd, page, dti, dt, norm, rope, pad = APPEND[i]
    S = Batch(100 + i, seqs, n_q, n_kv, hd, page, dt, pad)
    qkv = dev(S.g.standard_normal((S.T, n_q + 2 * n_kv, hd), dtype=np.float32) * 2, dti)
    Q, K, V = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    gq = dev(1 + 0.1 * S.g.standard_normal(hd), dt) if norm else None
    gk = dev(1 + 0.1 * S.g.standard_normal(hd), dt) if norm else None
    f = (10000.0 ** (-2 * np.arange(hd // 2) / hd)).astype(np.float32) if rope else None
    Qo = torch.full((S.T, n_q, hd), 7.0, dtype=dt, device="cuda")
    K0, V0 = S.Kp.clone(), S.Vp.clone()
    out = B.dllm_paged_append(K, V, S.Kp, S.Vp, *S.d, Q=Q, Q_out=Qo, gamma_q=gq, gamma_k=gk, eps=1e-6,
                              inv_freq=None if f is None else torch.from_numpy(f).cuda())
    assert out is Qo
    h = {n: None if t is None else host(t) for n, t in (("q", gq), ("k", gk))}
    Kr, Vr, Qr, lost = paged.append(host(K), host(V), host(K0), host(V0), S.table, S.q_start, S.kv_len, Q=host(Q),
                                    Q_out=np.full((S.T, n_q, hd), 7.0), gamma_q=h["q"], gamma_k=h["k"], eps=1e-6,
                                    inv_freq=f)
    assert lost == 0 and B.check_status() == 0
    changed = (Kr != host(K0)).any((2, 3)) | (Vr != host(V0)).any((2, 3))
    assert changed.sum() == sum(n for n, _ in seqs)
    for got, ref, before in ((S.Kp, Kr, K0), (S.Vp, Vr, V0)):
        same = torch.from_numpy(~changed).cuda()
        assert torch.equal(got[same], before[same])       # other slots: bit for bit
    assert torch.equal(Qo[S.rows:], torch.full_like(Qo[S.rows:], 7.0))
    assert np.abs(host(S.Vp) - Vr)[changed].max() <= U[dt] * np.abs(Vr[changed]).max()
    for got, ref in ((host(S.Kp)[changed], Kr[changed]), (host(Qo)[:S.rows], Qr[:S.rows])):
        pair = np.hypot(ref[..., :hd // 2], ref[..., hd // 2:])
        tol = U[dt] * np.abs(ref) + 2e-6 * np.concatenate([pair, pair], -1)
        assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) - tol)


def test_append_keys_alone_in_place_queries_and_layer_table(B):
    S = Batch(7, [(9, 20), (2, 2)], 4, 2, 64, 16, F32)
    K, V, Q = (dev(S.g.standard_normal((S.T, h, 64), dtype=np.float32), F32) for h in (2, 2, 4))
    assert B.dllm_paged_append(K, V, S.Kp, S.Vp, *S.d) is None
    Kr, Vr, _, _ = paged.append(host(K), host(V), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len)
    assert np.array_equal(host(S.Kp), Kr) and np.array_equal(host(S.Vp), Vr)
    w = {n: torch.zeros(s, device="cuda") for n, s in (("w_q", (256, 64)), ("w_k", (128, 64)), ("w_v", (128, 64)),
                                                       ("w_o", (64, 256)), ("w_g", (64, 64)), ("w_u", (64, 64)),
                                                       ("w_d", (64, 64)), ("gamma1", (64,)), ("gamma2", (64,)))}
    layer = B.dllm_pack_layer(w, 4, 2, 64)
    ref = B.dllm_paged_append(K, V, S.Kp, S.Vp, *S.d, Q=Q, inv_freq=layer)
    Qi = Q.clone()
    assert B.dllm_paged_append(K, V, S.Kp, S.Vp, *S.d, Q=Qi, Q_out=Qi, inv_freq=layer) is Qi
    assert torch.equal(Qi, ref)
    f = (10000.0 ** (-2 * np.arange(32) / 64)).astype(np.float32)
    _, _, Qr, _ = paged.append(host(K), host(V), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, Q=host(Q),
                               Q_out=np.zeros((S.T, 4, 64)), inv_freq=f)
    assert np.abs(host(ref) - Qr).max() <= 2e-6 * np.abs(Qr).max() * 2


def test_append_rows_without_a_page_raise_the_status(B):
    S = Batch(8, [(10, 20), (4, 40), (5, 3)], 1, 1, 64, 8, F32, max_pages=4)
    table = S.table.copy()
    table[0, 1] = S.P                                  # outside the pool: positions 10 .. 15 lost
    d = [torch.from_numpy(table).cuda(), *S.d[1:]]     # sequence 1: positions 36 .. 39 past the table
    K, V, Q = (dev(S.g.standard_normal((S.T, 1, 64), dtype=np.float32), F32) for _ in range(3))
    Kb, Vb = host(S.Kp), host(S.Vp)
    Qo = torch.full((S.T, 1, 64), 3.0, device="cuda")
    B.dllm_paged_append(K, V, S.Kp, S.Vp, *d, Q=Q, Q_out=Qo)
    Kr, Vr, Qr, lost = paged.append(host(K), host(V), Kb, Vb, table, S.q_start, S.kv_len, Q=host(Q),
                                    Q_out=np.full((S.T, 1, 64), 3.0))
    assert lost == 10
    assert B.check_status(reset=True) == B.STATUS_PAGE
    assert np.array_equal(host(S.Kp), Kr) and np.array_equal(host(S.Vp), Vr) and np.array_equal(host(Qo), Qr)
    assert (host(Qo)[14:16] == 3.0).all()              # before position 0: skipped


# ---------------------------------------------------------------------------- attention
ATTEND = [
    # seqs (new, keys), n_q, n_kv, hd, page, mask_block, pad
    ([(1, 1)], 1, 1, 64, 8, 0, 0),
    ([(32, 1024)], 4, 4, 128, 64, 0, 0),
    ([(1, 77), (1, 16), (1, 3000), (1, 1), (1, 129)], 28, 4, 128, 16, 1, 3),
    ([(1, 5000)] * 3, 8, 1, 128, 16, 0, 0),
    ([(67, 130), (0, 0), (5, 5), (33, 4097), (0, 9)], 6, 2, 64, 32, 1, 4),
    ([(300, 700), (129, 129), (1, 300)], 7, 1, 128, 128, 32, 0),
    ([(256, 256), (255, 511)], 2, 2, 64, 256, 1, 1),
    ([(5, 3), (4, 0), (2, 2), (3, 200)], 4, 2, 128, 16, 1, 2),       # rows before position 0
    ([(5, 3), (4, 0), (2, 2)], 4, 2, 64, 8, 0, 0),
    ([(40, 640)], 128, 1, 64, 64, 7, 0),                             # 128 heads share a key head
    ([(2, 1000), (18, 2100)], 100, 2, 128, 32, 0, 0),
    ([(600, 1300)], 2, 1, 128, 64, 1, 0),
]


def check_attention(got, lse, ref, S, dt, scale=None, live=None):
    A, Aa, L, n = ref
    live = np.arange(S.T) < S.rows if live is None else live
    Qn = np.linalg.norm(host(S.Q), axis=-1)
    kmax = np.nanmax(np.linalg.norm(host(S.Kp), axis=-1)) if S.P else 0.0
    sc = scale or S.hd ** -0.5
    ds = S.hd * 2.0 ** -23 * Qn * kmax * sc
    rel = 2 * ds[..., None] + n[:, None, None] * 2.0 ** -23 + 1e-5
    tol = U[dt] * np.abs(A) + Aa * (rel + (U[BF] if dt == BF else 0.0)) * 1.01 + 1e-30
    err = np.abs(host(got) - A)
    assert np.isfinite(host(got)[live]).all()
    assert (err[live] <= tol[live]).all(), (err - tol)[live].max()
    if lse is not None:
        l = host(lse)[live]
        assert np.array_equal(np.isneginf(l), np.isneginf(L[live]))
        ok = np.isfinite(L[live])
        lt = (ds + n[:, None] * 2.0 ** -23 + 1e-5 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0)))[live]
        assert (np.abs(l[ok] - L[live][ok]) <= lt[ok]).all()


def attend_case(B, i, dt):
    seqs, n_q, n_kv, hd, page, mb, pad = ATTEND[i]
    S = Batch(300 + i, seqs, n_q, n_kv, hd, page, dt, pad)
    S.poison()
    S.Q = dev(S.g.standard_normal((S.T, n_q, hd), dtype=np.float32) * 1.5, dt)
    A = torch.full((S.T, n_q, hd), 5.0, dtype=dt, device="cuda")
    lse = torch.full((S.T, n_q), 5.0, device="cuda")
    out = B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, max(n for n, _ in seqs), mask_block=mb, A=A, lse=lse)
    assert out is A and B.check_status() == 0
    assert (A[S.rows:] == 5.0).all() and (lse[S.rows:] == 5.0).all()      # padded rows: as they were
    ref = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, mb)
    check_attention(A, lse, ref, S, dt)
    return S, A


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attention_parity(B, i, dt):
    attend_case(B, i, dt)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_attention_absent_pages_and_short_tables(B, dt):
    """Entries outside the pool and keys past the table are absent; a row with none gets zeros."""
    S = Batch(40, [(3, 90), (2, 40), (35, 300), (1, 10)], 4, 2, 64, 16, dt, max_pages=10)
    table = S.table.copy()
    table[0, 1], table[0, 3] = -1, S.P
    table[1, :] = -5
    table[2, :9] = 1 << 30
    S.table = table
    S.d[0] = torch.from_numpy(table).cuda()
    S.poison()
    S.Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), dt)
    for mb in (0, 1):
        lse = torch.empty((S.T, 4), device="cuda")
        A = B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 35, mask_block=mb, lse=lse)
        ref = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), table, S.q_start, S.kv_len, mb)
        assert (ref[3] == 0).any() and (ref[3] > 0).any()
        check_attention(A, lse, ref, S, dt)
        assert not host(A)[ref[3] == 0].any()
    assert B.check_status() == 0


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_attention_climbing_maxima_strided_queries_and_scale(B, dt):
    """Scores that grow along the keys by far more than an exponent's range, at another scale,
    with the queries a strided slice; the largest key decides."""
    hd, n = 64, 900
    S = Batch(41, [(2, n), (40, n)], 4, 2, hd, 32, dt)
    ramp = np.linspace(-40, 40, n).astype(np.float32)
    kv = np.zeros((2, n, 2, hd), np.float32)
    kv[:, :, :, 0] = ramp[None, :, None]
    for b in range(2):
        for j in range(n):
            S.Kp[S.table[b, j // 32], j % 32] = torch.from_numpy(kv[b, j]).to(dt)
    wide = dev(S.g.standard_normal((S.T, 7, hd), dtype=np.float32), dt)
    wide[:, 1:5, 0] = 30.0
    S.Q = wide[:, 1:5]
    A = B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 40, mask_block=0, scale=0.25)
    ref = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, 0, 0.25)
    check_attention(A, None, ref, S, dt, 0.25)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_attention_repeats_bit_for_bit_and_replays_new_lengths(B, dt):
    """The same inputs give the same bits; a captured call follows lengths, tables and rows that
    are rewritten between replays, on a side stream."""
    S, A = attend_case(B, 4, dt)
    for _ in range(3):
        again = B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 67, mask_block=1)
        assert torch.equal(again[:S.rows], A[:S.rows])
    out = torch.zeros_like(A)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 67, mask_block=1, A=out)
    B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 67, mask_block=0)      # (other work in between)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:S.rows], A[:S.rows])
    kv = S.kv_len.copy()
    kv[3] -= 1000
    kv[2] = 2
    starts = S.q_start.copy()
    starts[1:4] -= 30                       # 37 rows in the first sequence, 63 in the fourth
    S.kv_len, S.q_start = kv, starts
    S.d[1].copy_(torch.from_numpy(starts))
    S.d[2].copy_(torch.from_numpy(kv))
    g.replay()
    torch.cuda.synchronize()
    ref = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), S.table, starts, kv, 1)
    check_attention(out, None, ref, S, dt)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_rows_outside_the_bounds_are_left_alone(B, dt):
    """Rows past max_new, rows of a sequence that reaches past T, and descending starts: computed
    where they are inside, untouched where not; a batch without any row and a call without rows."""
    S = Batch(42, [(50, 400), (3, 90), (20, 700)], 4, 2, 64, 16, dt)
    S.Q = dev(S.g.standard_normal((S.T, 4, 64), dtype=np.float32), dt)
    ref = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, 1)
    for most in (1, 7, 33, 49):
        A = torch.full((S.T, 4, 64), 9.0, dtype=dt, device="cuda")
        B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, most, mask_block=1, A=A)
        slot = np.concatenate([np.arange(n) for n, _ in S.seqs])
        inside = torch.from_numpy(slot < most).cuda()
        assert (A[~inside] == 9.0).all() and not (A[inside] == 9.0).all(-1).any()
        check_attention(A, None, ref, S, dt, live=slot < most)
    # the last sequence's rows reach past T; the one before has descending starts
    starts = np.array([0, 50, 40, 80], np.int32)
    T = 60
    A = torch.full((T, 4, 64), 9.0, dtype=dt, device="cuda")
    lse = torch.full((T, 4), 9.0, device="cuda")
    d1 = torch.from_numpy(starts).cuda()
    B.dllm_paged_attention(S.Q[:T], S.Kp, S.Vp, S.d[0], d1, S.d[2], 50, mask_block=1, A=A, lse=lse)
    assert torch.isfinite(A).all() and (A[50:] != 9.0).any()
    Qo = torch.full((T, 4, 64), 9.0, dtype=dt, device="cuda")
    kv = torch.zeros((T, 2, 64), dtype=dt, device="cuda")
    B.dllm_paged_append(kv, kv, S.Kp, S.Vp, S.d[0], d1, S.d[2], Q=S.Q[:T], Q_out=Qo)
    torch.cuda.synchronize()
    # no rows at all
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    A = torch.full((5, 4, 64), 9.0, dtype=dt, device="cuda")
    B.dllm_paged_attention(S.Q[:5], S.Kp, S.Vp, S.d[0], zero, S.d[2], 5, A=A)
    assert (A == 9.0).all()
    e = torch.empty((0, 4, 64), dtype=dt, device="cuda")
    assert B.dllm_paged_attention(e, S.Kp, S.Vp, S.d[0], zero, S.d[2], 5).shape == (0, 4, 64)
    assert B.dllm_paged_append(e[:, :2], e[:, :2], S.Kp, S.Vp, S.d[0], zero, S.d[2], Q=e).shape == (0, 4, 64)
    assert B.check_status(reset=True) in (0, B.STATUS_PAGE)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_as_many_sequences_as_a_batch_may_have(B, dt):
    """1024 sequences, a third of them without a new row and a few without a key: append, then attend."""
    g = synth.rng(43)
    seqs = [(0 if b % 3 == 1 else 1 + b % 4, 0) for b in range(1024)]
    seqs = [(n, n + (0 if b % 7 == 0 else int(g.integers(0, 150)))) for b, (n, _) in enumerate(seqs)]
    S = Batch(44, seqs, 6, 2, 64, 8, dt)
    K, V, Q = (dev(S.g.standard_normal((S.T, h, 64), dtype=np.float32), dt) for h in (2, 2, 6))
    Qo = B.dllm_paged_append(K, V, S.Kp, S.Vp, *S.d, Q=Q)
    assert torch.equal(Qo, Q)
    kp, vp = host(S.Kp), host(S.Vp)
    for b in (0, 2, 500, 1022, 1023):
        for i in range(seqs[b][0]):
            pos, row = seqs[b][1] - seqs[b][0] + i, S.q_start[b] + i
            p = S.table[b, pos // 8]
            assert np.array_equal(kp[p, pos % 8], host(K)[row]) and np.array_equal(vp[p, pos % 8], host(V)[row])
    S.Q = Qo
    lse = torch.empty((S.T, 6), device="cuda")
    A = B.dllm_paged_attention(Qo, S.Kp, S.Vp, *S.d, 4, mask_block=1, lse=lse)
    check_attention(A, lse, paged.attention(host(Qo), kp, vp, S.table, S.q_start, S.kv_len, 1), S, dt)
    assert B.check_status() == 0


def test_streams_and_graphs_do_not_share_scratch(B):
    """Calls on two streams at once, and two captured graphs replayed side by side, each give what
    they give alone."""
    runs = []
    for i, (seqs, mb) in enumerate((([(1, 3000)] * 9, 0), ([(200, 900), (64, 2000)], 1))):
        S = Batch(80 + i, seqs, 8, 2, 128, 32, BF)
        S.Q = dev(S.g.standard_normal((S.T, 8, 128), dtype=np.float32), BF)
        most = max(n for n, _ in seqs)
        call = lambda A, S=S, most=most, mb=mb: B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, most, mask_block=mb, A=A)  # noqa: E731
        runs.append((call, call(torch.empty_like(S.Q)), torch.empty_like(S.Q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for call, want, out, st in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call(out)
        graphs.append(g)
    for use_graph in (False, True):
        for _, _, out, _ in runs:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for (call, _, out, st), g in zip(runs, graphs):
                with torch.cuda.stream(st):
                    g.replay() if use_graph else call(out)
        torch.cuda.synchronize()
        for _, want, out, _ in runs:
            assert torch.equal(out, want)
    assert B.check_status() == 0


def test_f32_sums_do_not_drift_over_a_long_cache(B):
    """65536 keys whose values share a mean: a running sum that rounds one way would move with their number."""
    S = Batch(45, [(2, 65536), (1, 30001)], 2, 1, 64, 64, F32)
    S.Vp += 1.0
    S.Q = dev(S.g.standard_normal((S.T, 2, 64), dtype=np.float32), F32)
    A = host(B.dllm_paged_attention(S.Q, S.Kp, S.Vp, *S.d, 2, mask_block=1))
    A0 = paged.attention(host(S.Q), host(S.Kp), host(S.Vp), S.table, S.q_start, S.kv_len, 1)[0]
    # relative to the outputs' norm: weights and values are split to 2^-21 each and their low parts'
    # product (2^-22) left out; 24 sums within a tile, 2^-23 each; a score of up to about 6 is off by
    # as much, which moves the weights by 6 times that, of either sign
    assert np.linalg.norm(A - A0) <= (2 * 2.0 ** -21 + 2.0 ** -22 + 24 * 2.0 ** -23) * 1.5 * np.linalg.norm(A0)


def test_attention_of_consecutive_pages_is_the_dense_attention(B):
    """A dense cache is a paged one with consecutive entries: both kernels answer alike."""
    Bn, N, n_q, n_kv, hd, k = 2, 512, 8, 4, 128, 48
    g = synth.rng(60)
    K, V = (dev(g.standard_normal((Bn, N, n_kv, hd), dtype=np.float32), BF) for _ in range(2))
    Q = dev(g.standard_normal((Bn * k, n_q * hd), dtype=np.float32), BF)
    idx = torch.arange(N, dtype=torch.int32).repeat(Bn, 1).cuda()
    cnt = torch.full((Bn,), k, dtype=torch.int32).cuda()
    dense = host(B.dllm_attention(Q, K, V, idx, cnt, k))
    table = torch.arange(Bn * N // 64, dtype=torch.int32).view(Bn, -1).cuda()
    qs = torch.tensor([0, k, 2 * k], dtype=torch.int32).cuda()
    kl = torch.full((Bn,), N, dtype=torch.int32).cuda()
    pg = host(B.dllm_paged_attention(Q.view(-1, n_q, hd), K.view(-1, 64, n_kv, hd), V.view(-1, 64, n_kv, hd), table,
                                     qs, kl, k)).reshape(dense.shape)
    # each side rounds its weights and its output to bf16 (A_abs <= max |v| ~ 5 is far above what
    # 512 near-uniform weights leave: the mean |v| of 0.8 bounds A_abs here)
    assert np.abs(dense - pg).max() <= 2 * 2.0 ** -8 * (np.abs(dense).max() + 1.0)


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_writes_stay_inside_their_arrays(B, dt):
    from test_gpu_guards import Guarded
    seqs = [(33, 100), (1, 4000), (130, 130)]
    S = Batch(50, seqs, 6, 2, 128, 16, dt, pad=2)
    G = Guarded(51)
    Kp, Vp = G.new(S.Kp.shape, dt, S.Kp), G.new(S.Vp.shape, dt, S.Vp)
    d = [G.new(t.shape, torch.int32, t) for t in S.d]
    Q, K, V = (G.new((S.T, h, 128), dt, torch.randn((S.T, h, 128)).to(dt)) for h in (6, 2, 2))
    Qo, A, lse = G.new((S.T, 6, 128), dt), G.new((S.T, 6, 128), dt), G.new((S.T, 6), F32)
    ws = G.new((max(16, B.dllm_paged_attention_workspace_bytes(S.T, 3, 130, 6, 2, 128, dt)),), torch.uint8)
    B.dllm_paged_append(K, V, Kp, Vp, *d, Q=Q, Q_out=Qo)
    for mb in (0, 1):
        B.dllm_paged_attention(Qo, Kp, Vp, *d, 130, mask_block=mb, A=A, lse=lse, ws=ws)
    assert B.check_status() == 0
    G.check()


def test_decode_block_by_block_over_pages(B):
    """The three operators as a server runs them: two sequences of different length grow by a block
    and then by single tokens; each step appends, attends over all pages, projects to a
    small vocabulary and samples.  Every step is checked against the definitions on the
    device's own inputs of that step."""
    n_q, n_kv, hd, page, V = 4, 2, 64, 16, 512
    lens = [37, 90]
    S = Batch(70, [(0, 260), (0, 260)], n_q, n_kv, hd, page, BF, scale=0.0)
    g = S.g
    W = dev(g.standard_normal((V, n_q * hd), dtype=np.float32) * 0.3, BF)
    f = (10000.0 ** (-2 * np.arange(hd // 2) / hd)).astype(np.float32)
    ft = torch.from_numpy(f).cuda()
    gq, gk = (dev(1 + 0.1 * g.standard_normal(hd), BF) for _ in range(2))
    table = S.d[0]
    for step, new in enumerate(([37, 90], [32, 32], [1, 1], [1, 1])):
        if step:
            lens = [l + n for l, n in zip(lens, new)]
        qs_h, kl_h = np.concatenate([[0], np.cumsum(new)]).astype(np.int32), np.array(lens, np.int32)
        qs, kl = torch.from_numpy(qs_h).cuda(), torch.from_numpy(kl_h).cuda()
        T = int(qs_h[-1])
        qkv = dev(g.standard_normal((T, n_q + 2 * n_kv, hd), dtype=np.float32), F32)
        Kb, Vb = host(S.Kp), host(S.Vp)
        Q, K, Vv = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        q = B.dllm_paged_append(K, Vv, S.Kp, S.Vp, table, qs, kl, Q=Q, gamma_q=gq, gamma_k=gk, inv_freq=ft)
        Kr, Vr, Qr, lost = paged.append(host(K), host(Vv), Kb, Vb, S.table, qs_h, kl_h, Q=host(Q), Q_out=np.zeros(q.shape),
                                        gamma_q=host(gq), gamma_k=host(gk), inv_freq=f)
        assert lost == 0
        for got, ref in ((host(q), Qr), (host(S.Kp), Kr), (host(S.Vp), Vr)):
            assert np.abs(got - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-5
        A = B.dllm_paged_attention(q, S.Kp, S.Vp, table, qs, kl, max(new), mask_block=1)
        S.Q, S.T, S.rows = q, T, T
        check_attention(A, None, paged.attention(host(q), host(S.Kp), host(S.Vp), S.table, qs_h, kl_h, 1), S, BF)
        last = torch.from_numpy(qs_h[1:].astype(np.int64) - 1).cuda()
        logits = B.dllm_gemm_bf16(A.view(T, -1)[last].contiguous(), W).view(2, 1, V)
        u = torch.from_numpy(g.random((2, 1)).astype(np.float32)).cuda()
        prm = dict(temperature=torch.tensor([0.7, 1.0], device="cuda"), top_p=torch.tensor([0.9, 1.0], device="cuda"),
                   top_k=torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
        tok, prob = B.dllm_sample(logits, u, **prm)
        lh, uh = logits.cpu().numpy(), u.cpu().numpy()
        for b in range(2):
            t, p = paged.sample_row(lh[b, 0], uh[b, 0], [0.7, 1.0][b], [0, 20][b], [0.9, 1.0][b])
            assert int(tok[b, 0]) == t and float(prob[b, 0]) == pytest.approx(p, rel=1e-6)
    assert B.check_status() == 0
