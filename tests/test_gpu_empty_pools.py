"""Caches with a pool that is there but holds no pages (a tier that is not in use): the calls are the same as
without it."""
import pytest
import torch

from paged_long_context_b200 import binding, synth
from tests._gpu import check, run
from tests._tree import TreeCall, tree_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


ROOM = []


def add_empty_pools(pool):
    """Pointers to pools of no pages, as a caller of the C ABI passes them for tiers that are not in use."""
    if not ROOM:
        ROOM.append(torch.zeros((1 << 16,), dtype=torch.uint8, device="cuda"))
    for f in (synth.BF16, synth.I8):
        if not pool.k_pool[f]:
            pool.k_pool[f] = pool.v_pool[f] = ROOM[0].data_ptr()
            pool.pool_pages[f] = 0


@pytest.mark.parametrize("Q", [3, 40])
@pytest.mark.parametrize("form", [dict(fmt="i8", P=64), dict(fmt="i4", P=16, d=64), dict(fmt="tiered", P=16, tiers=[(0.5, "i4"), (0.5, "fp8")])],
                         ids=["i8", "i4-d64", "i4-fp8"])
def test_tree_attention(form, Q):
    case = tree_case((700, 41, 130), Q, **form)
    call = TreeCall(case)
    add_empty_pools(call.pool)
    assert call.run() == 0
    call.check()
    assert int(call.err.item()) == 0


def test_tree_attention_of_pages_in_an_empty_pool():
    # bf16 pages are named, none is there: every token is left out and reported
    case = tree_case((50, 130), 3, fmt="bf16")
    call = TreeCall(case)
    call.pool.pool_pages[synth.BF16] = 0
    assert call.run() == 0
    torch.cuda.synchronize()
    assert int(call.err.item()) == binding.DEVERR_PAGE_ID
    assert (call.out == 0).all() and torch.isneginf(call.lse).all()


@pytest.mark.parametrize("form", [dict(fmt="i8", P=64), dict(fmt="i4", P=16), dict(fmt="fp8", P=64), dict(fmt="i8", P=16, d=64)],
                         ids=["i8", "i4", "fp8", "i8-d64"])
def test_decode(form, monkeypatch):
    case = tree_case((700, 41, 130), 1, **form)
    assert binding.decode_path(case) == 2
    plain = binding.kv_pool_struct

    def with_empty_pools(c):
        pool = plain(c)
        add_empty_pools(pool)
        return pool

    monkeypatch.setattr(binding, "kv_pool_struct", with_empty_pools)
    assert binding.decode_path(case) == 2
    out, lse, err = run(case)
    check(case, out, lse, host_case=case.to("cpu"))
    assert err == 0
