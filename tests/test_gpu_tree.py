"""Attention of a tree of drafted tokens over the paged cache (cfr_paged_decode_tree)
against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding, synth
from tests._tree import TreeCall, chain, random_tree, tree_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


def trees(B, Q, seed):
    rng = np.random.default_rng(seed)
    both = [random_tree(Q, rng) for _ in range(B)]
    return [m for m, _ in both], [d for _, d in both]


TIERS = [(0.3, "i4"), (0.3, "i8"), (0.2, "fp8"), (0.2, "bf16")]
CONFIGS = {
    "bf16-p16": dict(),
    "bf16-p16-d64": dict(d=64),
    "bf16-p128": dict(P=128),
    "bf16-p512": dict(P=512),
    "bf16-p24": dict(P=24),
    "bf16-p16-formats-given": dict(use_page_fmt=True),
    "bf16-mha": dict(Hq=4, Hkv=4),
    "bf16-mqa": dict(Hq=9, Hkv=1),
    "i8-p16": dict(fmt="i8"),
    "i8-p256": dict(fmt="i8", P=256),
    "i4-p32": dict(fmt="i4", P=32),
    "i4-p24-d64": dict(fmt="i4", P=24, d=64),
    "fp8-p64": dict(fmt="fp8", P=64),
    "fp8-p8-d64": dict(fmt="fp8", P=8, d=64),
    "tiered-p16": dict(fmt="tiered", tiers=TIERS),
    "tiered-p128": dict(fmt="tiered", tiers=TIERS, P=128),
    "tiered-p256-d64": dict(fmt="tiered", tiers=TIERS, P=256, d=64),
    "f32-p16": dict(fmt="f32", q_fmt="f32"),
    "f32-mixed": dict(fmt="tiered", tiers=[(0.5, "f32"), (0.5, "i8")], d=64),
    "f32-q-on-bf16": dict(q_fmt="f32"),
}
# lengths where a tile, a page or the prefix ends: alone, at a border, one off it
LENS = (5, 127, 128, 129, 133, 700, 1537)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(CONFIGS))
def test_random_trees(name, out_dtype):
    case = tree_case(LENS, 5, **CONFIGS[name])
    masks, depths = trees(len(LENS), 5, 11)
    call = TreeCall(case, masks, depths, out_dtype=out_dtype)
    assert call.run() == 0
    call.check()
    assert int(call.err.item()) == 0


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p128", "i8-p16", "f32-p16", "bf16-p24"])
@pytest.mark.parametrize("cap", [0.0, 3.0, 50.0])
def test_alibi_depths_and_cap(name, cap):
    case = tree_case(LENS, 5, alibi=True, **CONFIGS[name])
    masks, depths = trees(len(LENS), 5, 12)
    call = TreeCall(case, masks, depths, cap=cap)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p256-d64", "i4-p32", "f32-p16"])
@pytest.mark.parametrize("Q", [1, 2, 17, 63, 64])
def test_numbers_of_drafts(name, Q):
    lens = (Q, Q + 1, 130 + Q, 300)
    case = tree_case(lens, Q, **CONFIGS[name])
    masks, depths = trees(len(lens), Q, 13)
    call = TreeCall(case, masks, depths)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "i8-p256", "f32-p16"])
def test_ragged_drafts_leave_other_rows_alone(name):
    lens, q_lens = (140, 3, 260, 9, 1), [0, 3, 9, 4, 1]
    case = tree_case(lens, 9, **CONFIGS[name])
    masks, depths = trees(len(lens), 9, 14)
    call = TreeCall(case, masks, depths, q_lens=q_lens)
    assert call.run() == 0
    call.check()
    assert int(call.err.item()) == 0


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p16", "f32-p16"])
def test_rows_that_see_nothing(name):
    # a sequence of drafts only, some of which see no token, not even themselves
    lens = (6, 150)
    case = tree_case(lens, 6, **CONFIGS[name])
    masks = [[0, 1, 0b100, 0, 0b11111, 0b100001], [0] * 6]   # the second sees its prefix only
    call = TreeCall(case, masks)
    assert call.run() == 0
    call.check()
    assert torch.isneginf(call.lse[0, 0]).all() and (call.out[0, 3] == 0).all()


def test_bits_behind_the_drafts_are_ignored():
    case = tree_case((40, 200), 5)
    masks, depths = trees(2, 5, 15)
    a = TreeCall(case, masks, depths, q_lens=[3, 4])
    b = TreeCall(case, [[m | 0xFF00000000000000 | (1 << 4) for m in row] for row in masks], depths, q_lens=[3, 4])
    assert a.run() == 0 and b.run() == 0
    torch.cuda.synchronize()
    assert torch.equal(a.out[:, :3], b.out[:, :3]) and torch.equal(a.lse[:, :3], b.lse[:, :3])


def test_no_mask_is_a_chain_and_agrees_with_multi_query_decode():
    case = tree_case((700, 77, 300), 4, alibi=True)
    call = TreeCall(case, out_dtype=torch.float32)
    assert call.run() == 0
    call.check()
    bufs = binding.paged_decode(case)
    torch.cuda.synchronize()
    a, b = call.out.view(3, 32, 128), bufs.out
    # two roundings of p to 16 bits apart, of values up to about 4
    assert (a - b).abs().max() <= 2 * 2.0 ** -8 * 4
    assert (call.lse.view(3, 32) - bufs.lse).abs().max() <= 1e-4


@pytest.mark.parametrize("name", ["bf16-p16", "i8-p16", "f32-p16"])
def test_head_map(name):
    case = tree_case(LENS, 5, head_map=[2, 0, 0, 2, 2, 2, 0, 2], **{**CONFIGS[name], "Hkv": 3})
    masks, depths = trees(len(LENS), 5, 16)
    call = TreeCall(case, masks, depths)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name,hq,hkv,Q", [("bf16-p16", 32, 2, 40), ("i8-p256", 16, 1, 33), ("bf16-p16", 64, 8, 64)])
def test_many_rows_of_one_kv_head(name, hq, hkv, Q):
    lens = (Q, 900)
    case = tree_case(lens, Q, **{**CONFIGS[name], "Hq": hq, "Hkv": hkv})
    masks, depths = trees(2, Q, 17)
    call = TreeCall(case, masks, depths)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p128"])
def test_many_sequences(name):
    lens = [1 + (i * 37) % 150 + 3 for i in range(300)]
    case = tree_case(lens, 2, Hq=2, Hkv=1, **{k: v for k, v in CONFIGS[name].items()})
    call = TreeCall(case)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "bf16-p24", "fp8-p64", "f32-p16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_drafts_reach_only_rows_that_see_them(name, bad):
    Q, n = 4, 260
    case = tree_case((n,), Q, **CONFIGS[name])
    f, P = case.uniform_fmt, case.page_tokens
    if f == synth.FP8 and np.isinf(bad):
        pytest.skip("E4M3 has no infinities")
    j = n - 3                                           # draft 1
    masks = [[0b0001, 0b0011, 0b0101, 0b1011]]          # drafts 1 and 3 see it
    call = TreeCall(case, masks)
    slot, row = int(case.page_table[0, j // P]), j % P
    for pool in (case.k_pool, case.v_pool):
        if f == synth.FP8:
            pool[f][slot, :, row, 5] = 0x7F
        else:
            view = pool[f].view(torch.float32 if f == synth.F32 else torch.bfloat16)
            view[slot, :, row, 5] = bad
    assert call.run() == 0
    call.check(skip={(0, i, h) for i in (1, 3) for h in range(8)})
    out = call.out.float().cpu()
    if np.isnan(bad):
        assert torch.isnan(out[0, [1, 3]]).all()


def test_infinite_value_with_finite_score():
    # V alone is infinite: the element that holds it is infinite in rows that see it, the others are finite
    Q, n = 3, 200
    case = tree_case((n,), Q)
    j = n - 2
    view = case.v_pool[synth.BF16].view(torch.bfloat16)
    view[int(case.page_table[0, j // 16]), :, j % 16, 9] = float("inf")
    call = TreeCall(case, [[0b001, 0b011, 0b101]])
    assert call.run() == 0
    call.check(skip={(0, 1, h) for h in range(8)})
    out = call.out[0, 1].float().cpu()
    assert torch.isposinf(out[:, 9]).all()
    out[:, 9] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p16", "f32-p16"])
def test_bad_pages_are_skipped_and_reported(name):
    case = tree_case((200, 90), 3, **CONFIGS[name])
    P = case.page_tokens
    case.page_table[0, 2] = 10 ** 6
    case.page_table[1, 0] = -4
    masks, depths = trees(2, 3, 18)
    call = TreeCall(case, masks, depths)
    assert call.run() == 0
    torch.cuda.synchronize()
    assert int(call.err.item()) == binding.DEVERR_PAGE_ID
    case.page_table[0, 2] = 0    # (readable again for the reference, which leaves the tokens out)
    case.page_table[1, 0] = 0
    call.check(dropped={(0, j) for j in range(2 * P, 3 * P)} | {(1, j) for j in range(P)})


def test_bad_formats_are_skipped_and_reported():
    case = tree_case((200,), 3, fmt="tiered", tiers=[(0.5, "i8"), (0.5, "bf16")])
    was = int(case.page_fmt[0, 1])
    for value, bit in ((9, binding.DEVERR_PAGE_FMT), (synth.FP8, binding.DEVERR_POOL)):
        case.page_fmt[0, 1] = value
        call = TreeCall(case)
        assert call.run() == 0
        torch.cuda.synchronize()
        assert int(call.err.item()) == bit
        case.page_fmt[0, 1] = was
        call.check(dropped={(0, j) for j in range(16, 32)})


@pytest.mark.parametrize("name", ["bf16-p16", "f32-p16"])
def test_bad_lengths_give_empty_rows(name):
    case = tree_case((200, 90, 64, 70), 3, **CONFIGS[name])
    case.seq_lens[1] = 2                               # fewer tokens than drafts
    case.seq_lens[2] = 10 ** 6                         # more than the table holds
    call = TreeCall(case, q_lens=[3, 3, 3, -1])
    assert call.run() == 0
    torch.cuda.synchronize()
    assert int(call.err.item()) == binding.DEVERR_SEQ_LEN
    assert (call.out[1:] == 0).all() and torch.isneginf(call.lse[1:]).all()
    assert torch.isfinite(call.out[0]).all()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p256-d64", "f32-p16"])
def test_repeats_are_equal_and_lse_may_be_absent(name):
    case = tree_case(LENS, 5, **CONFIGS[name])
    masks, depths = trees(len(LENS), 5, 19)
    calls = [TreeCall(case, masks, depths) for _ in range(3)]
    calls[2].lse = None
    for c in calls:
        assert c.run() == 0
    torch.cuda.synchronize()
    assert torch.equal(calls[0].out, calls[1].out) and torch.equal(calls[0].lse, calls[1].lse)
    assert torch.equal(calls[0].out, calls[2].out)


@pytest.mark.parametrize("name", ["bf16-p16", "i8-p256", "f32-p16"])
def test_captured_calls_and_two_streams(name):
    cases = [tree_case((900, 77, 310), 5, seed=s, **CONFIGS[name]) for s in (5, 6)]
    masks, depths = trees(3, 5, 20)
    calls = [TreeCall(c, masks, depths) for c in cases]
    want = []
    for c in calls:
        assert c.run() == 0
        torch.cuda.synchronize()
        want.append((c.out.clone(), c.lse.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    graphs = []
    for c, s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            assert c.run(stream=s) == 0
        graphs.append(g)
    for _ in range(3):
        for c in calls:
            c.out.zero_()
            c.lse.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):          # both at once, each with its own workspace
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, (o, l) in zip(calls, want):
            assert torch.equal(c.out, o) and torch.equal(c.lse, l)


def test_workspace_too_small_is_refused():
    case = tree_case((40,), 2)
    call = TreeCall(case)
    call.workspace = call.workspace[:-256]
    assert call.run() == binding.STATUS_CODES["CFR_ERR_WORKSPACE"]


def test_offsets_beyond_32_bits():
    # a pool of more than 2^32 bytes whose last pages are used
    d, hkv, P = 128, 8, 512
    pages = (1 << 32) // (hkv * P * d * 2) + 40
    k = torch.zeros((pages, hkv, P, 2 * d), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    case = tree_case((1300,), 3, Hq=8, Hkv=hkv, P=P)
    ids = [pages - 1, pages - 30, 1]
    for new, old in zip(ids, case.page_table[0].tolist()):
        k[new] = case.k_pool[synth.BF16][old]
        v[new] = case.v_pool[synth.BF16][old]
    want = TreeCall(case)
    assert want.run() == 0
    case.k_pool[synth.BF16], case.v_pool[synth.BF16] = k, v
    case.page_table[0] = torch.tensor(ids, dtype=torch.int32)
    got = TreeCall(case)
    assert got.run() == 0
    torch.cuda.synchronize()
    assert torch.equal(want.out, got.out) and torch.equal(want.lse, got.lse)


# long enough for a CTA to walk many tiles of an item, several items and their borders
@pytest.mark.parametrize("Q", [3, 40], ids=["12rows", "160rows"])
@pytest.mark.parametrize("name", ["bf16-p16", "bf16-p16-d64", "bf16-p24", "i8-p16", "i8-p256", "i4-p32", "fp8-p8-d64", "tiered-p16",
                                  "tiered-p128", "tiered-p256-d64", "f32-p16"])
def test_long_sequences(name, Q):
    lens = (9001, 18303, 130, 5120)
    cfg = {**CONFIGS[name], "Hq": 8, "Hkv": 2}
    case = tree_case(lens, Q, **cfg)
    masks, depths = trees(len(lens), Q, 21)
    call = TreeCall(case, masks, depths, q_lens=[Q, Q - 1, Q, Q // 2])
    assert call.run() == 0
    call.check()
    assert int(call.err.item()) == 0
    again = TreeCall(case, masks, depths, q_lens=[Q, Q - 1, Q, Q // 2])
    assert again.run() == 0
    torch.cuda.synchronize()
    assert torch.equal(again.out, call.out) and torch.equal(again.lse, call.lse)


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p128", "f32-p16"])
def test_scores_that_grow_along_the_sequence(name):
    # each tile's maximum passes the last one's by more than the step at which the running reference moves
    case = tree_case((9001, 2100), 3, softmax_scale=1.0, alibi=True, **CONFIGS[name])
    case.alibi_slopes[:] = torch.tensor([0.2, 0.11, 0.05, 0.02, 0.5, 1.0, 0.3, 0.07], device="cuda")
    call = TreeCall(case)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "i8-p16", "f32-p16"])
@pytest.mark.parametrize("cap", [1e-30, 2.0 ** -10, 700.0, 1024.0])
def test_small_and_large_caps(name, cap):
    case = tree_case(LENS, 5, **CONFIGS[name])
    masks, depths = trees(len(LENS), 5, 20)
    call = TreeCall(case, masks, depths, cap=cap)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p128", "f32-p16"])
@pytest.mark.parametrize("cap", [1e7, 3e38])
def test_caps_far_above_the_scores_change_nothing(name, cap):
    case = tree_case(LENS, 5, **CONFIGS[name])
    masks, depths = trees(len(LENS), 5, 21)
    call = TreeCall(case, masks, depths, cap=cap)
    assert call.run() == 0
    call.cap = 0.0    # a score of 30 is 1e-10 off under a cap of 1e7: the formula's and the bounds without one
    call.check()


@pytest.mark.parametrize("name", ["bf16-p16", "tiered-p128", "f32-p16"])
@pytest.mark.parametrize("cap,lean", [(30.0, -1.0), (55.0, -1.0), (55.0, 1.0), (55.0, 0.0), (60.0, -1.0)])
def test_scores_at_both_ends_of_the_cap(name, cap, lean):
    # queries so long that most scores stand at one end of the cap (all of them below, all above, or both)
    case = tree_case((133, 700), 5, **CONFIGS[name])
    call = TreeCall(case, *trees(2, 5, 22), cap=cap)
    if lean:
        if "tiered" in name:    # codes of one sign: each row's scores lean one way by the queries' sign
            for f in case.k_pool:
                if f == synth.BF16:
                    case.k_pool[f].copy_(case.k_pool[f].view(torch.bfloat16).abs().view(case.k_pool[f].dtype).view_as(case.k_pool[f]))
                elif f == synth.I8:
                    case.k_pool[f].bitwise_and_(0x3F)
                elif f == synth.I4:
                    case.k_pool[f].bitwise_and_(0x77)
                else:
                    case.k_pool[f].bitwise_and_(0x7F)
        else:
            dt = torch.float32 if name.startswith("f32") else torch.bfloat16
            for f in case.k_pool:
                k = case.k_pool[f].view(dt)
                k.copy_(k.abs())
        call.q.copy_(call.q.abs() * lean * 60)
    else:
        call.q.mul_(60)
    assert call.run() == 0
    call.check()
