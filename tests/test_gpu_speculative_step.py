"""A speculative step over the paged cache, as a decoder runs it: the drafts' queries and keys are
normed, rotated and appended, the tree is attended, and the accepted branch is moved to follow the
prefix by reading its rows back and writing them again; decoding then goes on from there."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding, synth
from tests._hostkv import host_kv
from tests._tree import BF16_HALF, F32_HALF, as_int64

pytestmark = pytest.mark.gpu

Q, HQ, HKV, D, P = 6, 8, 2, 128, 16
PARENTS = [-1, 0, 0, 1, 2, 2]
ACCEPTED = [0, 2, 5]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


def tree():
    masks, depths = [], []
    for i, p in enumerate(PARENTS):
        masks.append((masks[p] if p >= 0 else 0) | (1 << i))
        depths.append(depths[p] + 1 if p >= 0 else 0)
    return masks, depths


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attend(q, K, V):
    """softmax(q K^T / sqrt(d)) V in 64 bits, and sum_j p_j |v_j|."""
    s = K @ q / np.sqrt(D)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ V, p @ np.abs(V)


@pytest.mark.parametrize("fmt", ["bf16", "i8"])
def test_draft_verify_and_accept(fmt):
    prefix = [133, 40]
    B = len(prefix)
    # pages for the prefix and the drafts; the drafts' rows hold whatever was there
    spec = synth.CaseSpec("spec", B, HQ, HKV, D, P, seq_lens=[n + Q for n in prefix], fmt=fmt, spare_pages=2)
    case = synth.make_case(spec, 31, "cuda")
    pool = binding.kv_pool_struct(case)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((B * Q, HQ + 2 * HKV, D), generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    w = (1 + 0.1 * torch.randn((D,), generator=g)).cuda()
    masks, depths = tree()
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    q_out = torch.empty((B * Q, HQ, D), dtype=torch.bfloat16, device="cuda")
    pos = i32([n + x for n in prefix for x in depths])
    err = torch.zeros((1,), dtype=torch.int32, device="cuda")

    # the drafts' K and V into the cache: straight into hot pages, or through a step's own pages into int8 ones
    seq, tok = i32([b for b in range(B) for _ in range(Q)]), i32([n + i for n in prefix for i in range(Q)])
    if fmt == "bf16":
        to, table = pool, case.page_table
    else:
        hot_k = torch.zeros((B, HKV, P, D), dtype=torch.bfloat16, device="cuda")
        hot_v = torch.zeros_like(hot_k)
        to = binding.pool_struct(HKV, D, P, {synth.BF16: hot_k}, {synth.BF16: hot_v})
        table, tok = i32([[b] for b in range(B)]), i32([i for _ in range(B) for i in range(Q)])
    assert binding.qk_norm_rope_append(to, q, k, v, pos, inv, q_out, table, None, synth.BF16, seq, tok, q_weight=w,
                                       k_weight=w, err=err) == 0
    if fmt == "i8":
        off = i32([0, Q, 2 * Q])
        step = [torch.empty((B * Q, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        assert binding.read_kv(to, table, None, synth.BF16, off, i32([0, 0]), *step, err=err) == 0
        assert binding.write_kv(pool, case.page_table, None, synth.I8, off, i32(prefix), *step, err=err) == 0

    # the tree's attention
    out = torch.empty((B, Q, HQ, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, Q, HQ), device="cuda")
    ws = torch.empty((binding.tree_workspace_size(B, Q, HQ, HKV, D),), dtype=torch.uint8, device="cuda")
    t_mask = as_int64([masks] * B)
    call = lambda o, l, lens, n, qq, m: binding.paged_decode_tree(  # noqa: E731
        pool, qq, case.page_table, lens, o, l, ws, uniform_fmt=case.uniform_fmt, tree_mask=m, err=err)
    assert call(out, lse, case.seq_lens, Q, q_out.view(B, Q, HQ, D), t_mask) == 0
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    hc = case.to("cpu")
    qh = q_out.double().cpu().numpy().reshape(B, Q, HQ, D)
    for b in range(B):
        for h in range(HQ):
            K, V = host_kv(hc, b, h // (HQ // HKV))
            for i in range(Q):
                seen = [j < prefix[b] or bool((masks[i] >> (j - prefix[b])) & 1) for j in range(prefix[b] + Q)]
                o, A = attend(qh[b, i, h], K[seen], V[seen])
                off_by = np.abs(out[b, i, h].double().cpu().numpy() - o)
                # p and out are each rounded once to 16 bits; sums and scores in 32 (see tests/_tree.py)
                assert (off_by <= (BF16_HALF + 400 * F32_HALF * 16) * A + BF16_HALF * np.abs(o) * 1.01).all()

    # accept a branch: its rows follow the prefix
    rows = [torch.empty((B * Q, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert binding.read_kv(pool, case.page_table, None, case.uniform_fmt, i32([0, Q, 2 * Q]), i32(prefix), *rows, err=err) == 0
    pick = torch.tensor([b * Q + i for b in range(B) for i in ACCEPTED], device="cuda")
    n = len(ACCEPTED)
    kept = [r[pick].contiguous() for r in rows]
    assert binding.write_kv(pool, case.page_table, None, case.uniform_fmt, i32([0, n, 2 * n]), i32(prefix), *kept, err=err) == 0
    case.seq_lens.copy_(i32([x + n for x in prefix]))

    # the accepted leaf's query over the compacted cache sees what it saw in the tree
    leaf = q_out.view(B, Q, HQ, D)[:, ACCEPTED[-1]:ACCEPTED[-1] + 1].contiguous()
    out1, lse1 = torch.empty_like(leaf), torch.empty((B, 1, HQ), device="cuda")
    ws1 = torch.empty((binding.tree_workspace_size(B, 1, HQ, HKV, D),), dtype=torch.uint8, device="cuda")
    ws = ws1 if ws1.numel() > ws.numel() else ws
    assert call(out1, lse1, case.seq_lens, 1, leaf, None) == 0
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    hc = case.to("cpu")
    for b in range(B):
        for h in range(HQ):
            K, V = host_kv(hc, b, h // (HQ // HKV))
            o, A = attend(leaf[b, 0, h].double().cpu().numpy(), K, V)
            off_by = np.abs(out1[b, 0, h].double().cpu().numpy() - o)
            assert (off_by <= (BF16_HALF + 400 * F32_HALF * 16) * A + BF16_HALF * np.abs(o) * 1.01).all()
            if fmt == "bf16":
                # the same tokens in other places: two calls, each off by its own tolerance
                both = 2 * ((BF16_HALF + 400 * F32_HALF * 16) * A + BF16_HALF * np.abs(o) * 1.01)
                assert (np.abs(out1[b, 0, h].double().cpu().numpy() - out[b, ACCEPTED[-1], h].double().cpu().numpy()) <= both).all()


def test_arguments_of_another_device_are_refused():
    spec = synth.CaseSpec("dev", 1, 4, 2, 64, 16, seq_lens=[40])
    case = synth.make_case(spec, 3, "cuda")
    pool = binding.kv_pool_struct(case)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)       # on the host
    with pytest.raises(ValueError, match="current device"):
        binding.write_kv(pool, case.page_table, None, synth.BF16, i32([0, 4]), i32([0]), k, k)
