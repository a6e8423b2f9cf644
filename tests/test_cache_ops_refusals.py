"""What the cache-writing, read-back and tree-attention entry points refuse on the
host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from paged_long_context_b200 import binding, synth
from paged_long_context_b200 import build as build_mod

INVALID, UNSUP, OVERFLOW, CUDA, WORKSPACE = 1, 2, 3, 5, 7
BF16, F32, I8 = synth.BF16, synth.F32, synth.I8


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.lib()


def p(t):
    return ctypes.c_void_p(t.data_ptr())


BUF = torch.zeros((1 << 16,), dtype=torch.float32)
ODD = ctypes.c_void_p(BUF.data_ptr() + 4)


def pool(fmt="bf16", **over):
    case = synth.make_case(synth.CaseSpec("r", 2, 4, 2, 64, 16, seq_lens=[40, 17], fmt=fmt), 3, "cpu")
    s = binding.kv_pool_struct(case)
    s.keep = case
    for k, v in over.items():
        setattr(s, k, v)
    return s


def rope(L, pool_=None, **over):
    a = dict(kv=ctypes.byref(pool_ if pool_ is not None else pool()), table=p(BUF), mp=3, pf=None, uf=BF16, b=2, q=p(BUF), qs=256,
             k=p(BUF), ks=128, v=p(BUF), vs=128, f=BF16, n=4, hq=4, qw=None, kw=None, eps=1e-6, pos=p(BUF), inv=p(BUF), rot=64,
             il=0, out=p(BUF), seq=p(BUF), tok=p(BUF), err=None, s=None)
    a.update(over)
    return L.cfr_qk_norm_rope_append(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(seq=None), INVALID), (dict(tok=None), INVALID),
    (dict(pos=None), INVALID), (dict(inv=None), INVALID), (dict(q=ODD), INVALID), (dict(out=ODD), INVALID),
    (dict(qw=ODD), INVALID), (dict(qs=255), INVALID), (dict(ks=127), INVALID), (dict(vs=132), INVALID), (dict(vs=-128), INVALID),
    (dict(ks=1 << 62), INVALID), (dict(f=I8), INVALID), (dict(uf=I8), INVALID), (dict(uf=F32), INVALID), (dict(b=0), INVALID),
    (dict(mp=0), INVALID), (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=257, qs=1 << 16), UNSUP), (dict(rot=-16), INVALID),
    (dict(rot=24), UNSUP), (dict(rot=80), UNSUP), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(mp=1 << 28), OVERFLOW), (dict(b=1 << 20, mp=1 << 12), OVERFLOW),
    (dict(n=0), 0), (dict(n=0, q=None, out=None), 0)])
def test_rope_refusals(lib, over, code):
    assert rope(lib, **over) == code


def test_rope_needs_a_hot_pool(lib):
    assert rope(lib, pool("i8")) == INVALID
    assert rope(lib, pool(head_dim=96)) == UNSUP
    assert rope(lib, pool(page_tokens=4)) == UNSUP
    assert rope(lib, pool(num_kv_heads=0)) == INVALID


def chunk(fn, pool_=None, **over):
    a = dict(kv=ctypes.byref(pool_ if pool_ is not None else pool()), table=p(BUF), mp=3, pf=None, uf=BF16, b=2, off=p(BUF),
             starts=p(BUF), k=p(BUF), ks=128, v=p(BUF), vs=128, f=BF16, n=4, err=None, s=None)
    a.update(over)
    return fn(*a.values())


@pytest.mark.parametrize("name", ["cfr_write_kv", "cfr_read_kv"])
@pytest.mark.parametrize("over,code", [
    (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(off=None), INVALID), (dict(starts=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=ODD), INVALID), (dict(ks=120), INVALID), (dict(vs=130), INVALID),
    (dict(f=I8), INVALID), (dict(n=-1), INVALID), (dict(b=-1), INVALID), (dict(uf=9), INVALID), (dict(uf=I8), INVALID),
    (dict(mp=1 << 28), OVERFLOW), (dict(n=0, k=None, v=None), 0)])
def test_chunk_refusals(lib, name, over, code):
    assert chunk(getattr(lib, name), **over) == code


@pytest.mark.parametrize("name", ["cfr_write_kv", "cfr_read_kv"])
def test_chunk_pool_refusals(lib, name):
    fn = getattr(lib, name)
    q = pool("i8")
    q.scales[I8] = None
    assert chunk(fn, q, uf=I8) == INVALID
    q = pool()
    q.v_pool[BF16] = None
    assert chunk(fn, q) == INVALID
    q = pool()
    q.pool_pages[BF16] = 1 << 60
    assert chunk(fn, q) == OVERFLOW
    assert chunk(fn, pool(num_kv_heads=300)) == UNSUP


def tree(L, pool_=None, **over):
    a = dict(q=p(BUF), qf=BF16, kv=ctypes.byref(pool_ if pool_ is not None else pool()), table=p(BUF), mp=3, lens=p(BUF), b=2,
             pf=None, uf=BF16, hq=4, nq=2, ql=None, mask=None, dep=None, hm=None, sl=None, scale=0.0, cap=0.0, out=p(BUF), of=BF16,
             lse=None, ws=None, wsb=0, err=None, s=None)
    a.update(over)
    return L.cfr_paged_decode_tree(*a.values())


def hm(*v):
    t = torch.tensor(v, dtype=torch.int32)
    hm.keep.append(t)
    return p(t)


hm.keep = []


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(qf=I8), INVALID), (dict(kv=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(b=0), INVALID), (dict(uf=7), INVALID), (dict(uf=F32), INVALID), (dict(hq=3), INVALID),
    (dict(hq=0), INVALID), (dict(hq=258), UNSUP), (dict(nq=0), INVALID), (dict(nq=65), UNSUP), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(cap=-2.0), INVALID),
    (dict(cap=float("nan")), INVALID), (dict(cap=float("inf")), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID),
    (dict(of=I8), INVALID), (dict(hm=hm(0, 1, 2, 0)), INVALID), (dict(hm=hm(0, -1, 1, 0)), INVALID),
    (dict(mp=1 << 28), OVERFLOW), (dict(b=1 << 20, mp=1 << 12), OVERFLOW)])
def test_tree_refusals(lib, over, code):
    assert tree(lib, **over) == code


def test_workspace(lib):
    # (without a GPU the size cannot be known: the call fails all the same, and launches nothing)
    assert tree(lib) in (WORKSPACE, CUDA)
    for bad in ((0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 65, 4, 2, 64), (1, 1, 0, 2, 64), (1, 1, 4, 0, 64), (1, 1, 4, 2, 96)):
        assert binding.tree_workspace_size(*bad) == 0


def test_binding_checks_what_the_abi_cannot_see():
    pl = pool()
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.ones((2,), dtype=torch.int32)
    out, lse, ws = torch.zeros_like(q), torch.zeros((2, 3, 4)), torch.zeros((16,), dtype=torch.uint8)
    call = lambda **o: binding.paged_decode_tree(pl, **{**dict(q=q, page_table=table, seq_lens=lens, out=out, lse=lse,  # noqa: E731
                                                               workspace=ws), **o})
    for bad in (dict(q=q.half()), dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(page_table=table.long()), dict(seq_lens=lens[:1]),
                dict(out=out[:1]), dict(lse=lse.double()), dict(tree_mask=torch.zeros((2, 3), dtype=torch.int32)),
                dict(tree_mask=torch.zeros((2, 2), dtype=torch.int64)), dict(depths=torch.zeros((2,), dtype=torch.int32)),
                dict(alibi_slopes=torch.zeros((3,))), dict(workspace=None), dict(page_fmt=torch.zeros((2, 2), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    off, starts = torch.zeros((3,), dtype=torch.int32), torch.zeros((2,), dtype=torch.int32)
    for fn in (binding.write_kv, binding.read_kv):
        for bad in (dict(k=k.half()), dict(k=k[:, :1]), dict(k=k.transpose(0, 1)), dict(v=k.float()), dict(v=k[:4]),
                    dict(off=off[:2]), dict(starts=starts.long()), dict(k=torch.zeros((5, 2, 128), dtype=torch.bfloat16)[:, :, ::2])):
            a = {**dict(off=off, starts=starts, k=k, v=k), **bad}
            with pytest.raises(ValueError):
                fn(pl, table, None, BF16, a["off"], a["starts"], a["k"], a["v"])
    qq = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    ids, inv = torch.zeros((5,), dtype=torch.int32), torch.zeros((32,), dtype=torch.float64)
    good = dict(q=qq, k=k, v=k, rope_positions=ids, inv_freq=inv, q_out=torch.zeros_like(qq), page_table=table, page_fmt=None,
                uniform_fmt=BF16, seq_ids=ids, token_ids=ids)
    for bad in (dict(q=qq.half()), dict(k=k[:4]), dict(v=k.float()), dict(inv_freq=inv.float()), dict(rope_positions=None),
                dict(q_out=qq.float()), dict(seq_ids=ids[:2]), dict(q_weight=torch.zeros((32,))),
                dict(k_weight=torch.zeros((64,), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            binding.qk_norm_rope_append(pl, **{**good, **bad})


def test_pages_and_tables_that_32_bits_cannot_count(lib):
    for fn in (lib.cfr_write_kv, lib.cfr_read_kv):
        assert chunk(fn, pool(page_tokens=(1 << 24) + 8), mp=1) == UNSUP
    big = pool(page_tokens=1 << 20)
    big.pool_pages[BF16] = 1
    assert tree(lib, big, mp=2047) != OVERFLOW
    assert tree(lib, pool(page_tokens=(1 << 30) - 8), mp=2) == OVERFLOW
