"""Scratch of the paged attention and the sampling that the binding keeps: calls whose launches
may overlap or be interleaved do not share it."""
import threading

import numpy as np
import pytest

from sparse_kv_cache_rank_gb300 import synth
from test_abi import dl  # noqa: F401  (the library fixture)

torch = pytest.importorskip("torch")


def test_threads_streams_and_calls_have_their_own(dl, monkeypatch):  # noqa: F811
    """Host memory in place of the device's, and a made-up stream."""
    stream = [7]
    monkeypatch.setattr(dl, "_getdev", lambda: 0)
    monkeypatch.setattr(dl, "_rawstream", lambda d: stream[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: stream[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    get = lambda n=64, tag="paged_attention": dl._stream_workspace(n, "cpu", 0, tag)   # noqa: E731
    mine = get()
    assert get().data_ptr() == mine.data_ptr()                    # one thread's calls are in order on a stream
    assert get(tag="sample").data_ptr() != mine.data_ptr()
    other, done, leave = [], threading.Event(), threading.Event()

    def work():
        other.append(get())
        done.set()
        leave.wait(10)                                            # (alive while the first thread goes on)

    th = threading.Thread(target=work)
    th.start()
    assert done.wait(10)
    assert other[0].data_ptr() != mine.data_ptr() and get().data_ptr() == mine.data_ptr()
    leave.set()
    th.join()
    stream[0] = 8
    assert get().data_ptr() != mine.data_ptr()
    stream[0] = 7
    assert get(1000).numel() >= 1000 and get(64).numel() >= 1000
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    kept = [get() for _ in range(3)]
    assert len({t.data_ptr() for t in kept}) == 3


@pytest.mark.gpu
def test_threads_on_one_stream(dl):  # noqa: F811
    """Two threads on the default stream, each attending over batches of its own lengths and drawing tokens of its
    own vocabulary: every call gives what it gives alone."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_paged import BF, Batch, dev
    runs = []
    for i, (seqs, V) in enumerate((([(1, 3000)] * 9, 20011), ([(200, 900), (64, 2000), (5, 9000)], 50021))):
        S = Batch(90 + i, seqs, 8, 2, 128, 32, BF)
        Q = dev(S.g.standard_normal((S.T, 8, 128), dtype=np.float32), BF)
        l = dev(synth.rng(95 + i).standard_normal((3, 2, V), dtype=np.float32) * 3, BF)
        u = torch.from_numpy(synth.rng(97 + i).random((3, 2)).astype(np.float32)).cuda()
        k = torch.full((3,), 40, dtype=torch.int32, device="cuda")
        most = max(n for n, _ in seqs)
        call = lambda S=S, Q=Q, l=l, u=u, k=k, most=most: (  # noqa: E731
            dl.dllm_paged_attention(Q, S.Kp, S.Vp, *S.d, most, mask_block=1), *dl.dllm_sample(l, u, top_k=k))
        runs.append((call, call()))
    torch.cuda.synchronize()
    start, right, wrong = threading.Barrier(2), [], []

    def work(call, want):
        start.wait(30)
        for _ in range(60):
            outs = [call() for _ in range(4)]
            for got in outs:
                (right if all(torch.equal(g, w) for g, w in zip(got, want)) else wrong).append(1)

    threads = [threading.Thread(target=work, args=r) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len(right) == 2 * 60 * 4 and dl.check_status() == 0


def test_sampling_of_a_small_vocabulary_needs_next_to_none(dl):  # noqa: F811
    """Up to 4096 tokens a row is one launch that keeps everything on the chip, however many rows."""
    L = dl.lib()
    assert [L.dllm_sample_workspace_bytes(*s) for s in ((1, 1, 1), (1, 20000, 12), (64, 1 << 10, 4096))] == [256] * 3
    assert L.dllm_sample_workspace_bytes(1, 20000, 4097) > 20000 * 4096


@pytest.mark.gpu
@pytest.mark.parametrize("V", [12, 4096])
def test_small_vocabularies_leave_their_scratch_alone(dl, V):  # noqa: F811
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    l = torch.from_numpy(synth.rng(V).standard_normal((2, 300, V), dtype=np.float32)).cuda()
    u = torch.from_numpy(synth.rng(V + 1).random((2, 300)).astype(np.float32)).cuda()
    p = torch.tensor([0.9, 1.0], device="cuda")
    ws = torch.full((256,), 171, dtype=torch.uint8, device="cuda")
    got = dl.dllm_sample(l, u, top_p=p, ws=ws)
    want = dl.dllm_sample(l, u, top_p=p)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (ws == 171).all()
    assert (got[0] >= 0).all() and (got[0] < V).all()
