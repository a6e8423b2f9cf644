"""Calls with bad offsets or lengths: what is in order is done in full, and nothing else is touched."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding
from tests._tree import TreeCall, tree_case
from tests.test_gpu_cache_io import BF16, FP8, I4, I8, Cache, chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


def in_order(off, starts, b, rows, tokens):
    return 0 <= off[b] <= off[b + 1] <= rows and starts[b] >= 0 and starts[b] + off[b + 1] - off[b] <= tokens


def write_one(c, state, k, v, off, starts, b):
    """Sequence b's rows, alone, into `state`."""
    n = off[b + 1] - off[b]
    c.expect_write(state, k[off[b]:off[b + 1]], v[off[b]:off[b + 1]], [0] * (b + 1) + [n] * (c.B - b), starts)


@pytest.mark.parametrize("fmts", [[I8], [I4], [FP8], [BF16], [I8, BF16, FP8]], ids=["i8", "i4", "fp8", "bf16", "mixed"])
@pytest.mark.parametrize("off,starts", [([0, 30, 20], [0, 0]), ([0, 10, 61], [0, 0]), ([-1, 10, 20], [0, 0]), ([0, 10, 20], [-1, 0]),
                                        ([0, 10, 20], [0, 39]), ([5, 3, 20], [0, 0])])
def test_a_sequence_out_of_range(off, starts, fmts):
    c = Cache(2, 2, 64, 16, 3, fmts, seed=12)
    state = c.host()
    k, v = chunk(60, 2, 64, torch.bfloat16, 13)
    assert c.write(k, v, off, starts) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN
    good = [b for b in range(2) if in_order(off, starts, b, 60, 48)]
    assert len(good) == 1
    write_one(c, state, k, v, off, starts, good[0])
    c.same(state)
    c.err.zero_()
    got = [torch.full((60, 2, 64), 9.0, device="cuda") for _ in range(2)]
    assert c.read(*got, off, starts) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN
    b = good[0]
    n = off[b + 1] - off[b]
    rows = c.expect_read([0] * (b + 1) + [n] * (c.B - b), starts, n, torch.float32)
    for a, r in zip(got, rows):
        want = torch.full((60, 2, 64), 9.0)
        want[off[b]:off[b + 1]] = r
        assert torch.equal(a.cpu(), want)


@pytest.mark.parametrize("fmt", [I8, I4, FP8])
def test_offsets_that_fit_several_sequences(fmt):
    # out of order, so that one place in the line of pages fits several sequences: a page of one that is in order is
    # its own in full or untouched, scale and all
    off, starts = [0, 60, 0, 40, 3], [0, 5, 3, 0]
    c = Cache(4, 1, 64, 8, 8, [fmt], seed=22)
    k, v = chunk(60, 1, 64, torch.bfloat16, 23)
    before, alone = c.host(), c.host()
    good = [b for b in range(4) if in_order(off, starts, b, 60, 64)]
    assert good == [0, 2]
    for b in good:
        write_one(c, alone, k, v, off, starts, b)
    assert c.write(k, v, off, starts) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN
    after = c.host()
    for b in range(4):
        for p in range(8):
            slot = int(c.table[b, p])
            for w in range(2):
                now = after[w][fmt][slot], after[2][fmt][slot, :, w]
                same = [np.array_equal(now[0], s[w][fmt][slot]) and np.array_equal(now[1], s[2][fmt][slot, :, w]) for s in (before, alone)]
                assert same[0] or (b in good and same[1]), (b, p, w)
    got = [torch.full((60, 1, 64), 9.0, device="cuda") for _ in range(2)]
    assert c.read(*got, off, starts) == 0
    # rows 0 .. 39 are named by two sequences in order, 40 .. 59 by one: theirs or untouched
    for w, a in enumerate(got):
        a = a.cpu()
        choices = [torch.full((60, 1, 64), 9.0)]
        for b in good:
            n = off[b + 1] - off[b]
            x = torch.full((60, 1, 64), 9.0)
            x[off[b]:off[b + 1]] = c.expect_read([0] * (b + 1) + [n] * (c.B - b), starts, n, torch.float32)[w]
            choices.append(x)
        for r in range(60):
            assert any(torch.equal(a[r], x[r]) for x in choices), r


@pytest.mark.parametrize("Q", [3, 40], ids=["12rows", "160rows"])
@pytest.mark.parametrize("form", [dict(), dict(fmt="i8", P=64), dict(fmt="f32", q_fmt="f32")], ids=["bf16", "i8", "f32"])
def test_bad_lengths_leave_the_other_sequences_right(form, Q):
    case = tree_case((200, 90, 64, 70, 300), Q, Hq=4, Hkv=1, **form)
    right = case.seq_lens.clone()
    case.seq_lens[1] = Q - 1                           # fewer tokens than drafts
    case.seq_lens[2] = 10 ** 6                         # more than the table holds
    call = TreeCall(case, q_lens=[Q, Q, Q, -1, Q])
    assert call.run() == 0
    torch.cuda.synchronize()
    assert int(call.err.item()) == binding.DEVERR_SEQ_LEN
    assert (call.out[1:4] == 0).all() and torch.isneginf(call.lse[1:4]).all()
    case.seq_lens.copy_(right)
    call.q_lens = [Q] * 5
    call.check(skip={(b, i, h) for b in (1, 2, 3) for i in range(Q) for h in range(4)})


@pytest.mark.parametrize("Q", [3, 40], ids=["12rows", "160rows"])
@pytest.mark.parametrize("form", [dict(), dict(fmt="i8", P=64), dict(fmt="f32", q_fmt="f32")], ids=["bf16", "i8", "f32"])
def test_no_drafts_at_all(form, Q):
    # nothing to do, whatever the lengths say
    case = tree_case((200, 90), Q, Hq=4, Hkv=1, **form)
    case.seq_lens[0], case.seq_lens[1] = -5, 2 ** 31 - 1
    call = TreeCall(case, q_lens=[0, 0])
    assert call.run() == 0
    torch.cuda.synchronize()
    assert (call.out == 7).all() and (call.lse == 7).all() and int(call.err.item()) == 0
