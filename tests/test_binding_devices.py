"""Host tensors are refused by the binding wherever there is a CUDA device, whether or not the process has used it yet (their
addresses would reach a kernel)."""
import os
import subprocess
import sys

import pytest
import torch

from paged_long_context_b200 import binding, synth

BF16 = synth.BF16


def calls():
    """Calls with every argument of the right type and shape, on the host."""
    case = synth.make_case(synth.CaseSpec("r", 2, 4, 2, 64, 16, seq_lens=[40, 17], fmt="bf16"), 3, "cpu")
    pool = binding.kv_pool_struct(case)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k, q = torch.zeros((5, 2, 64), dtype=torch.bfloat16), torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    tq = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    return [
        lambda: binding.write_kv(pool, i32(2, 3), None, BF16, i32(3), i32(2), k, k.clone()),
        lambda: binding.read_kv(pool, i32(2, 3), None, BF16, i32(3), i32(2), k.clone(), k.clone()),
        lambda: binding.qk_norm_rope_append(pool, q, k, k.clone(), i32(5), torch.zeros((32,), dtype=torch.float64), torch.zeros_like(q),
                                            i32(2, 3), None, BF16, i32(5), i32(5)),
        lambda: binding.paged_decode_tree(pool, tq, i32(2, 3), i32(2), torch.zeros_like(tq), None, torch.zeros((1 << 20,), dtype=torch.uint8)),
    ]


def refused():
    for call in calls():
        with pytest.raises(ValueError, match="cuda:0, the current device"):
            call()


def test_host_tensors_before_the_device_was_used(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    refused()


@pytest.mark.gpu
def test_host_tensors_in_a_fresh_process():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    code = "import torch\nfrom tests import test_binding_devices as t\nassert not torch.cuda.is_initialized()\nt.refused()\n"
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
