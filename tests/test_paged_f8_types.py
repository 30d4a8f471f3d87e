"""A torch without the types of 8-bit pages loses the calls over them and no others (no GPU)."""
import os
import subprocess
import sys

import pytest

from test_abi import ROOT, dl  # noqa: F401  (the library fixture)

pytest.importorskip("torch")

PROGRAM = """
import torch
del torch.{gone}
from sparse_kv_cache_rank_gb300 import binding as B
assert B.dllm_layer_budget(0.25, 1024) == 256
u = torch.zeros((2, 16, 1, 64), dtype=torch.uint8)
e = torch.zeros((2, 1), dtype=torch.uint8)
t, qs, kl = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
x = torch.zeros((3, 1, 64))
for call in (lambda: B.dllm_paged_append_f8(x, x, u, u, e, e, t, qs, kl),
             lambda: B.dllm_paged_attention_f8(x.bfloat16(), u, u, e, e, t, qs, kl, 3)):
    try:
        call()
    except B.DllmError as err:
        assert "{gone}" in str(err), err
    else:
        raise AssertionError("taken")
try:
    B.dllm_paged_append(x, x, torch.zeros((2, 16, 1, 64)), torch.zeros((2, 16, 1, 64)), t, qs, kl)
except B.DllmError as err:
    assert "CUDA" in str(err), err          # as far as without a device
"""


@pytest.mark.parametrize("gone", ["float8_e8m0fnu", "float8_e4m3fn"])
def test_other_calls_do_without(dl, gone):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(gone=gone)], cwd=ROOT, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": ROOT}, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
