"""GPU parity of the attention over 8-bit pages where a row's weights differ by many orders, with many tiles of keys to
each stream of a CTA: one key far above all others (an attention sink) before, among or after thousands whose small weights
add up, and tiles that take turns at being the largest.  The reference is 64-bit arithmetic on the device.

Tolerance (u = half a step, relative: bf16 2^-8, fp16 2^-11, E4M3 2^-4) of an element A = sum_j x_j code_j, x_j = w_j 2^v_j / sum w:
the scores' error ds as in test_gpu_paged_f8.py, a weight exp(+-2 ds), 1e-5 for the exponential, u(fp16), u(E4M3)^2 = 2^-8
for its two parts or, of a small one, 2^-13 of the largest x in its tile of 128 keys (no more than 2^-17 and no less than 2^-41
of the row's, never more than itself); the output u |A|.
"""
import pytest

from test_gpu_paged import BF, B  # noqa: F401  (B: the library fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
E4M3, E8M0, F64 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float64

# sequences, new rows, keys of the longest, n_q, n_kv, hd, page, mask_block: the forms of up to 8, 16, 32, 64 and 128 rows
# of a key head; 8 to 40 tiles for each of 152 CTAs
FORMS = [
    (48, 1, 8000, 8, 2, 128, 16, 1),
    (40, 4, 7000, 6, 2, 64, 64, 0),
    (24, 30, 7900, 2, 2, 128, 256, 4),
    (30, 17, 6500, 4, 2, 64, 8, 1),
    (12, 70, 9000, 6, 3, 128, 32, 1),
    (25, 130, 8100, 3, 3, 64, 128, 0),
]


class Case:
    def __init__(self, i):
        self.nb, self.n, most, self.n_q, self.n_kv, self.hd, self.page, self.mb = FORMS[i]
        self.g = g = torch.Generator(device="cuda").manual_seed(500 + i)
        self.lens = [most - (97 * b) % 1500 for b in range(self.nb)]
        need = [-(-k // self.page) for k in self.lens]
        self.P = sum(need)
        ids = torch.randperm(self.P, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((self.nb, max(need)), -1, dtype=torch.int32, device="cuda")
        for b, m in enumerate(need):
            self.table[b, :m] = ids[sum(need[:b]):sum(need[:b]) + m]
        shape = (self.P, self.page, self.n_kv, self.hd)
        self.K = torch.randn(shape, generator=g, device="cuda") * 100
        self.V = torch.randn(shape, generator=g, device="cuda") * 100 + 50
        self.K[..., 0] = 0
        self.Ve = torch.full((self.P, self.n_kv), -7, device="cuda")
        # scores of N(0, 1) under scale 1 and key scales 2^-7, and what the first dim adds
        self.Q = torch.randn((self.nb * self.n, self.n_q, self.hd), generator=g, device="cuda") * 1.28 / self.hd ** 0.5

    def rows(self, b):
        """Pool rows (page, slot) of sequence b's keys, in order."""
        j = torch.arange(self.lens[b], device="cuda")
        return self.table[b].long()[j // self.page], j % self.page

    def attend(self, B):  # noqa: F811
        self.K, self.V, self.Q = self.K.clamp(-448, 448).to(E4M3), self.V.clamp(-448, 448).to(E4M3), self.Q.to(BF)
        u8 = lambda e: (e + 127).to(torch.uint8).view(E8M0)   # noqa: E731
        starts = torch.arange(self.nb + 1, dtype=torch.int32, device="cuda") * self.n
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        lse = torch.empty((self.nb * self.n, self.n_q), device="cuda")
        A = B.dllm_paged_attention_f8(self.Q, self.K, self.V, u8(torch.full_like(self.Ve, -7)), u8(self.Ve), self.table, starts,
                                      lens, self.n, mask_block=self.mb, scale=1.0, lse=lse)
        assert B.check_status() == 0 and torch.isfinite(A).all()
        return A, lse

    def check(self, A, lse):
        G, worst = self.n_q // self.n_kv, 0.0
        for b in range(self.nb):
            pg, at = self.rows(b)
            t = slice(b * self.n, (b + 1) * self.n)
            pos = self.lens[b] - self.n + torch.arange(self.n, device="cuda")
            end = torch.full_like(pos, self.lens[b]) if self.mb == 0 else ((pos // self.mb + 1) * self.mb).clamp(max=self.lens[b])
            dead = torch.arange(self.lens[b], device="cuda")[None, :] >= end[:, None]
            for h in range(self.n_q):
                K, V = self.K[pg, at, h // G].to(F64) * 2.0 ** -7, self.V[pg, at, h // G].to(F64)
                q = self.Q[t, h].to(F64)
                s = (q @ K.T).masked_fill(dead, -torch.inf)
                L = torch.logsumexp(s, 1, keepdim=True)
                x = torch.exp(s - L) * torch.exp2(self.Ve[pg, h // G].to(F64))
                ref, mag = x @ V, x @ V.abs()
                tiles = torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).unflatten(1, (-1, 128)).amax(2)
                row = x.amax(1, keepdim=True)
                f = torch.minimum(tiles.repeat_interleave(128, 1)[:, :x.shape[1]] * 2.0 ** -13, row * 2.0 ** -17)
                f = torch.minimum(torch.maximum(f, row * 2.0 ** -41), x)
                kn, k1 = K.norm(dim=1).max(), K.abs().sum(1).max()
                ds = (self.hd * 2.0 ** -23 * q.norm(dim=1) * kn + 2.0 ** -17 * q.abs().amax(1) * k1)[:, None]
                rel = 2 * ds + x.shape[1] * 2.0 ** -23 + 1e-5 + 2.0 ** -11 + 2.0 ** -8
                tol = 2.0 ** -8 * ref.abs() + 1.01 * (mag * rel + f @ V.abs())
                worst = max(worst, float(((A[t, h].to(F64) - ref).abs() / tol).max()))
                lt = ds + x.shape[1] * 2.0 ** -23 + 1e-5 + 2.0 ** -22 * L.abs()
                assert ((lse[t, h].to(F64)[:, None] - L).abs() <= lt).all()
        assert worst <= 1, worst


@pytest.mark.parametrize("height", [10, 13, 24])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_small_weights_behind_a_sink_add_up(B, i, where, height):  # noqa: F811
    """One key e^height above the others, its value and those of its tile 0: the result is the others'."""
    S = Case(i)
    for b in range(S.nb):
        pg, at = S.rows(b)
        j = {"first": 0, "middle": S.lens[b] // 2, "last": S.lens[b] - S.n}[where]
        S.K[pg[j], at[j]] = 0
        S.K[pg[j], at[j], :, 0] = 448
        S.V[pg[j // 128 * 128:j // 128 * 128 + 128], at[j // 128 * 128:j // 128 * 128 + 128]] = 0
    S.Q[..., 0] = height / 3.5
    S.check(*S.attend(B))


@pytest.mark.parametrize("spread", [0, 10])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_tiles_that_take_turns(B, i, spread):  # noqa: F811
    """Every tile of 128 keys has a level of its own, up to e^12 apart, with value scales against them."""
    S = Case(i)
    S.V -= 50
    for b in range(S.nb):
        pg, at = S.rows(b)
        level = torch.rand((-(-S.lens[b] // 128)), generator=S.g, device="cuda") * 256 - 128
        S.K[pg, at, :, 0] = level.repeat_interleave(128)[:S.lens[b], None]
    if spread:
        S.Ve += torch.randint(-spread, spread + 1, S.Ve.shape, generator=S.g, device="cuda")
    S.Q[..., 0] = 6.0
    S.Q[:, ::2, 0] = -4.0
    S.check(*S.attend(B))


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_values_at_both_ends_of_the_scales(B, i, late):  # noqa: F811
    """Pages of zeros (scale 2^-64) beside pages of scale 2^55 to 2^63, all keys with like scores: the zeros count in the
    sum of the weights."""
    S = Case(i)
    S.Ve = torch.randint(55, 64, S.Ve.shape, generator=S.g, device="cuda")
    for b in range(S.nb):
        p = torch.arange(-(-S.lens[b] // S.page), device="cuda")
        ids = S.table[b, :len(p)].long()[(p * S.page // 384 % 2 == 1) == late]
        S.V[ids] = 0
        S.Ve[ids] = -64
    S.check(*S.attend(B))
