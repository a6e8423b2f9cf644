"""Infinite values of drafts that rule the rows which see them: the element is infinite, the others are the draft's own."""
import pytest
import torch

from paged_long_context_b200 import synth
from tests._tree import TreeCall, tree_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 8, 22], ids=lambda h: f"{3 * h}rows")
@pytest.mark.parametrize("n", [67, 100, 131, 163, 195, 227, 700])   # drafts in each quarter of a tile
def test_a_ruling_draft(n, heads, fmt):
    Q = 3
    case = tree_case((n,), Q, Hq=heads, Hkv=1, softmax_scale=1.0, fmt=fmt, q_fmt=fmt)
    call = TreeCall(case, [[0b001, 0b010, 0b101]], out_dtype=torch.float32)
    j = n - 2                                         # draft 1, which its own row alone sees
    f = synth.F32 if fmt == "f32" else synth.BF16
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    slot, row = int(case.page_table[0, j // 16]), j % 16
    k, v = case.k_pool[f].view(dt), case.v_pool[f].view(dt)
    call.q[0, 1] = call.q[0, 1, :1]                   # (one query for all heads of the row)
    k[slot, 0, row] = 4 * call.q[0, 1, 0]             # a score some 400 above every other token's
    v[slot, 0, row, 9] = float("inf")
    v[slot, 0, row, 70] = float("-inf")
    assert call.run() == 0
    call.check(skip={(0, 1, h) for h in range(heads)})
    got, want = call.out[0, 1], v[slot, 0, row].float()
    assert torch.isposinf(got[:, 9]).all() and torch.isneginf(got[:, 70]).all()
    rest = [e for e in range(128) if e not in (9, 70)]
    # other weights are below 2^-100: the sum's 2^-22 and half a step of fp32 remain
    assert ((got[:, rest] - want[rest]).abs() <= 2.0 ** -20 * want[rest].abs()).all()
