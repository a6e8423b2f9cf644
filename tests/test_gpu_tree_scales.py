"""Tree attention over quantised pages whose V scales differ by large factors, with and without a cap, against the
formula in 64 bits: what a page's scale does to its probabilities must not reach the softmax's sums."""
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


FORMS = {"i8-p256": dict(fmt="i8", P=256), "i8-p16": dict(fmt="i8", P=16), "i4-p64": dict(fmt="i4", P=64), "fp8-p128-d64": dict(fmt="fp8", P=128, d=64),
         "i8-fp8-p128": dict(fmt="tiered", P=128, tiers=[(0.5, "i8"), (0.5, "fp8")])}
LENS = (700, 133)


def set_scales(case, newest, older, k_newest=1.0):
    """V scales of the page that holds a sequence's last token, and of its other pages; a factor on the former's K scales."""
    for b, n in enumerate(case.seq_lens.tolist()):
        last = (n - 1) // case.page_tokens
        for p in range(last + 1):
            f = case.uniform_fmt if case.page_fmt is None else int(case.page_fmt[b, p])
            slot = int(case.page_table[b, p])
            case.scales[f][slot, :, 1] = newest if p == last else older
            if p == last:
                case.scales[f][slot, :, 0] *= k_newest


def one_sign(case):
    for f in case.k_pool:
        case.k_pool[f].bitwise_and_({synth.I8: 0x3F, synth.I4: 0x77, synth.FP8: 0x7F}[f])


# (newest, older): alike, within a few powers of two, and far apart either way
SCALES = [(0.01, 0.02), (1.0, 2.0 ** -14), (2.0 ** -6, 2.0 ** -21), (1.0, 2.0 ** -30), (2.0 ** 16, 2.0 ** -20), (1.0, 2.0 ** 30), (2.0 ** -18, 4.0),
          (2.0 ** 18, 2.0 ** 17)]


@pytest.mark.parametrize("Q", [3, 33], ids=["6rows", "66rows"])
@pytest.mark.parametrize("scales", SCALES, ids=lambda s: "%g-%g" % s)
@pytest.mark.parametrize("cap,lean", [(50.0, -60.0), (55.0, -60.0), (55.0, 60.0), (30.0, 1.0)])
@pytest.mark.parametrize("name", list(FORMS))
def test_capped_scores_at_the_ends(name, cap, lean, scales, Q):
    case = tree_case(LENS, Q, Hq=2, Hkv=1, **FORMS[name])
    one_sign(case)
    set_scales(case, *scales)
    call = TreeCall(case, cap=cap, out_dtype=torch.float32)
    call.q.copy_(call.q.abs() * lean)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("Q", [3, 33], ids=["6rows", "66rows"])
@pytest.mark.parametrize("scales", SCALES + [(2.0 ** 19, 2.0 ** -96), (1.0, 2.0 ** -90), (2.0 ** 30, 2.0 ** -60)], ids=lambda s: "%g-%g" % s)
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (0.0, True), (80.0, False)])
@pytest.mark.parametrize("name", list(FORMS))
def test_a_ruling_token_beside_many_light_ones(name, cap, alibi, scales, Q):
    # one score is some ten above hundreds of others, whose weights together are no less
    case = tree_case(LENS, Q, Hq=2, Hkv=1, alibi=alibi, **FORMS[name])
    if alibi:
        case.alibi_slopes[:] = torch.tensor([1e-3, 1e-4], device="cuda")
    set_scales(case, *scales, k_newest=3.0)
    call = TreeCall(case, cap=cap, out_dtype=torch.float32)
    assert call.run() == 0
    call.check()
