"""Tree attention where every CTA walks many items: large and small trees in turn, far more of them than the
kernel keeps item descriptions, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding, synth
from tests._tree import TreeCall, chain, tree_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


def repeated(call, copies):
    """The call's sequences `copies` times over (the same pages, the same queries): outputs by copy."""
    c = call.case
    B, Q, H, d = call.out.shape
    again = lambda t: None if t is None else t.repeat((copies,) + (1,) * (t.dim() - 1)).contiguous()  # noqa: E731
    out = torch.full((B * copies, Q, H, d), 7.0, dtype=call.out.dtype, device="cuda")
    lse = torch.full((B * copies, Q, H), 7.0, device="cuda")
    ws = torch.empty((binding.tree_workspace_size(B * copies, Q, H, c.num_kv_heads, d),), dtype=torch.uint8, device="cuda")
    st = binding.paged_decode_tree(
        call.pool, again(call.q), again(c.page_table), again(c.seq_lens), out, lse, ws, page_fmt=again(c.page_fmt),
        uniform_fmt=c.uniform_fmt, q_lens=again(call.t_q_lens), tree_mask=again(call.t_mask), softmax_scale=c.softmax_scale,
        logit_cap=call.cap, err=call.err)
    assert st == 0
    torch.cuda.synchronize()
    assert int(call.err.item()) == 0
    return out.view(copies, B, Q, H, d), lse.view(copies, B, Q, H)


def check_all(call, out, lse, skip=()):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref = call.reference()
    for b in range(out.shape[1]):
        for i in range(out.shape[2]):
            for h in range(out.shape[3]):
                if (b, i) in skip:
                    continue
                if (b, i, h) not in ref:
                    assert (out[:, b, i, h] == 7.0).all() and (lse[:, b, i, h] == 7.0).all()
                    continue
                o, l, to, tl = ref[b, i, h]
                assert (np.abs(out[:, b, i, h] - o) <= to).all() and (np.abs(lse[:, b, i, h] - l) <= tl).all(), (b, i, h)


TIERS = [(0.5, "i8"), (0.5, "bf16")]
# heads of 64 and of 128, each format; four query heads of a kv head: 64 drafts are 256 rows, 32 are 128, 33 are 132
FORMS = {"bf16-p16": dict(), "bf16-p16-d64": dict(d=64), "i8-p16": dict(fmt="i8"), "fp8-p64-d64": dict(fmt="fp8", P=64, d=64),
         "tiered-p16": dict(fmt="tiered", tiers=TIERS), "tiered-p16-d64": dict(fmt="tiered", tiers=TIERS, d=64)}


@pytest.mark.parametrize("copies", [40, 300])
@pytest.mark.parametrize("name", list(FORMS))
def test_large_and_small_trees_in_turn(name, copies):
    lens, q_lens = (70, 5, 90, 33, 140, 66, 40, 300), [64, 3, 33, 32, 1, 64, 8, 16]
    case = tree_case(lens, 64, Hq=4, Hkv=1, **FORMS[name])
    call = TreeCall(case, q_lens=q_lens)
    check_all(call, *repeated(call, copies))


@pytest.mark.parametrize("name", list(FORMS))
def test_small_trees_only(name):
    lens, q_lens = (12, 5, 140, 33), [9, 3, 16, 5]
    case = tree_case(lens, 16, Hq=4, Hkv=1, **FORMS[name])
    call = TreeCall(case, q_lens=q_lens)
    check_all(call, *repeated(call, 600))


@pytest.mark.parametrize("name", ["bf16-p16", "bf16-p16-d64", "fp8-p64-d64", "tiered-p16"])
def test_values_added_back_beside_many_small_trees(name):
    # drafts whose V is not finite, seen by rows of the second row tile only, then small trees
    lens, q_lens = (70, 5, 9, 33, 12, 20, 7, 30, 6, 8, 10, 40), [64] + [3, 5, 1, 7, 4, 2, 8, 3, 4, 5, 6]
    case = tree_case(lens, 64, Hq=4, Hkv=1, **FORMS[name])
    call = TreeCall(case, [chain(64)[0]] * len(lens), q_lens=q_lens)
    P, f = case.page_tokens, case.uniform_fmt
    first = 48
    for i in range(first, 64):
        j = lens[0] - 64 + i
        if case.page_fmt is not None:
            f = int(case.page_fmt[0, j // P])
            assert f == synth.BF16
        slot = int(case.page_table[0, j // P])
        if f == synth.FP8:
            case.v_pool[f][slot, :, j % P, i] = 0x7F
        else:
            case.v_pool[f].view(torch.bfloat16)[slot, :, j % P, i] = float("nan")
    out, lse = repeated(call, 200)
    check_all(call, out, lse, skip={(0, i) for i in range(first, 64)})
    for i in range(first, 64):   # element e is NaN in the rows from draft e on
        got = torch.isnan(out[:, 0, i])
        assert got[..., first:i + 1].all() and not got[..., :first].any() and not got[..., i + 1:].any()


@pytest.mark.parametrize("Q", [3, 40], ids=["12rows", "160rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_stretches_of_bf16_tiles_in_a_tiered_cache(d, Q):
    # most tiles need no expansion, and most stretches of a long sequence hold nothing else; the newest pages are coded
    case = tree_case((20000, 9001, 130), Q, Hq=4, Hkv=1, d=d, P=16, fmt="tiered", tiers=[(0.9, "bf16"), (0.1, "fp8")])
    call = TreeCall(case, q_lens=[Q, Q - 1, Q])
    P = case.page_tokens
    j = 20000 - 2
    f, slot = int(case.page_fmt[0, j // P]), int(case.page_table[0, j // P])
    assert f == synth.FP8
    case.v_pool[f][slot, :, j % P, 5] = 0x7F
    assert call.run() == 0
    call.check(skip={(0, i, h) for i in (Q - 2, Q - 1) for h in range(4)})
    got = torch.isnan(call.out[0, Q - 2:])
    assert got[..., 5].all() and not got[..., :5].any() and not got[..., 6:].any()
    assert int(call.err.item()) == 0
