"""Chunks of new tokens written into pages of every format (cfr_write_kv) and read
back (cfr_read_kv): bytes, scales and values against the definition, computed
page by page on the host."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding, synth
from tests._hostkv import decode_rows

pytestmark = pytest.mark.gpu
F32, BF16, I8, I4, FP8 = synth.F32, synth.BF16, synth.I8, synth.I4, synth.FP8
QMAX = {I8: 127.0, I4: 7.0, FP8: 448.0}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


def encode(x, fmt, scale):
    """Stored bytes of fp32 rows x [n][d], by the definition (fp32 quotient, ties to even)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    if fmt == F32:
        return x.view(np.uint8)
    if fmt == BF16:
        return torch.from_numpy(x).to(torch.bfloat16).view(torch.uint8).numpy()
    with np.errstate(all="ignore"):
        q = x / np.float32(scale) if scale > 0 else np.zeros_like(x)
    if fmt == FP8:
        t = torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        t[np.isnan(q)] = 0x7F
        return t
    r = np.clip(np.rint(np.where(np.isnan(q), 0, q)), -QMAX[fmt], QMAX[fmt]).astype(np.int8)
    if fmt == I8:
        return r.view(np.uint8)
    n = r.view(np.uint8) & 15
    return n[:, 0::2] | (n[:, 1::2] << 4)


class Cache:
    """A cache of random bytes, its tables on the GPU and a copy of its pools on the host."""

    def __init__(self, B, Hkv, d, P, pages, fmts, seed=0):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.P, self.pages = B, Hkv, d, P, pages
        self.fmt = rng.choice(fmts, size=(B, pages)).astype(np.uint8)
        self.table = np.zeros((B, pages), np.int32)
        self.k, self.v, self.scales = {}, {}, {}
        for f in set(fmts):
            where = np.argwhere(self.fmt == f)
            slots = rng.permutation(len(where) + 2)
            for (b, p), s in zip(where, slots):
                self.table[b, p] = s
            n = len(slots)
            for pool in (self.k, self.v):
                x = torch.from_numpy(rng.standard_normal((n, Hkv, P, d), dtype=np.float32))
                if f == F32:
                    pool[f] = x.view(torch.uint8).cuda()
                elif f == BF16:
                    pool[f] = x.to(torch.bfloat16).view(torch.uint8).cuda()
                else:
                    raw = rng.integers(0, 256, (n, Hkv, P, synth.row_bytes(f, d)), dtype=np.uint8)
                    raw[(raw & 0x7F) == 0x7F] = 0x11
                    pool[f] = torch.from_numpy(raw).cuda()
            if f in QMAX:
                self.scales[f] = torch.from_numpy(rng.uniform(0.5, 3, (n, Hkv, 2)).astype(np.float32) / np.float32(QMAX[f])).cuda()
        self.uniform = fmts[0] if len(set(fmts)) == 1 else None
        self.t_table = torch.from_numpy(self.table).cuda()
        self.t_fmt = None if self.uniform is not None else torch.from_numpy(self.fmt).cuda()
        self.pool = binding.pool_struct(Hkv, d, P, self.k, self.v, self.scales)
        self.err = torch.zeros((1,), dtype=torch.int32, device="cuda")

    def args(self):
        return self.pool, self.t_table, self.t_fmt, self.uniform if self.uniform is not None else 0

    def host(self):
        return ({f: t.cpu().numpy().copy() for f, t in self.k.items()}, {f: t.cpu().numpy().copy() for f, t in self.v.items()},
                {f: t.cpu().numpy().copy() for f, t in self.scales.items()})

    def write(self, k, v, off, starts):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        st = binding.write_kv(*self.args(), i32(off), i32(starts), k, v, err=self.err)
        torch.cuda.synchronize()
        return st

    def read(self, k, v, off, starts):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        st = binding.read_kv(*self.args(), i32(off), i32(starts), k, v, err=self.err)
        torch.cuda.synchronize()
        return st

    def expect_write(self, state, k, v, off, starts):
        """Applies the chunk to `state` (host pools and scales)."""
        pools, scales, P = state[:2], state[2], self.P
        for b in range(self.B):
            n, s = off[b + 1] - off[b], starts[b]
            for p in range(s // P, -(-(s + n) // P) if n else s // P):
                lo, hi = max(s, p * P), min(s + n, p * P + P)
                f, slot = int(self.fmt[b, p]), int(self.table[b, p])
                for w, rows in enumerate((k, v)):
                    for g in range(self.Hkv):
                        x = rows[off[b] + lo - s:off[b] + hi - s, g].float().cpu().numpy()
                        page = pools[w][f][slot, g]
                        scale = np.float32(1)
                        if f in QMAX:
                            finite = np.abs(x[~np.isnan(x)])
                            scale = np.float32(finite.max() if finite.size else 0) / np.float32(QMAX[f])
                            old = scales[f][slot, g, w]
                            if lo > p * P:
                                scale = max(scale, old)
                                if scale != old:
                                    kept = decode_rows(page[:lo - p * P].copy(), f, self.d).astype(np.float32) * old
                                    page[:lo - p * P] = encode(kept, f, scale)
                            scales[f][slot, g, w] = scale
                        page[lo - p * P:hi - p * P] = encode(x, f, scale)

    def same(self, state):
        for w, pool in enumerate((self.k, self.v)):
            for f in pool:
                assert np.array_equal(pool[f].cpu().numpy(), state[w][f]), (w, f)
        for f in self.scales:
            assert np.array_equal(self.scales[f].cpu().numpy(), state[2][f]), f

    def expect_read(self, off, starts, rows, dtype):
        out = [torch.full((rows, self.Hkv, self.d), 9.0, dtype=dtype) for _ in range(2)]
        pools = self.k, self.v
        for b in range(self.B):
            for r in range(off[b], off[b + 1]):
                j = starts[b] + r - off[b]
                f, slot = int(self.fmt[b, j // self.P]), int(self.table[b, j // self.P])
                for w in range(2):
                    raw = pools[w][f][slot, :, j % self.P].cpu().numpy()
                    x = decode_rows(raw, f, self.d).astype(np.float32)
                    if f in QMAX:
                        x = x * self.scales[f][slot, :, w].cpu().numpy()[:, None]
                    out[w][r] = torch.from_numpy(x).to(dtype)
        return out


def chunk(rows, Hkv, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return tuple((torch.randn((rows, Hkv, d), generator=g) * scale).to(dtype).cuda() for _ in range(2))


FORMATS = [[F32], [BF16], [I8], [I4], [FP8], [F32, BF16, I8, I4, FP8]]
# (page, first tokens, lengths): page borders hit, missed by one, chunks inside one page, none at all
SHAPES = [(16, [0, 5, 16, 31, 7], [1, 1, 16, 2, 0]),
          (8, [3, 0, 8, 15, 1], [40, 8, 0, 1, 23]),
          (24, [0, 23, 24, 1, 47], [24, 26, 47, 0, 3]),
          (256, [0, 255, 100, 256, 1], [256, 2, 300, 5, 254])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"p{s[0]}" for s in SHAPES])
@pytest.mark.parametrize("fmts", FORMATS, ids=lambda f: "-".join(synth.FMT_NAMES[x] for x in f))
def test_write_and_read(fmts, shape, dtype):
    P, starts, lens = shape
    d = 64 if dtype == torch.float32 else 128
    B, Hkv, pages = len(lens), 3, 8 if P < 256 else 3
    off = [0] + np.cumsum(lens).tolist()
    c = Cache(B, Hkv, d, P, pages, fmts, seed=P)
    state = c.host()
    for step, scale in enumerate((1.0, 3.0, 0.2)):    # a larger chunk grows the scales, a smaller one does not
        k, v = chunk(off[-1], Hkv, d, dtype, step, scale)
        assert c.write(k, v, off, starts) == 0
        c.expect_write(state, k, v, off, starts)
        c.same(state)
    back = [max(0, s - 3) for s in starts]
    lens2 = [s + n - a for s, n, a in zip(starts, lens, back)]
    off2 = [0] + np.cumsum(lens2).tolist()
    for out_dtype in (torch.float32, torch.bfloat16):
        got = [torch.full((off2[-1] + 2, Hkv, d), 9.0, dtype=out_dtype, device="cuda") for _ in range(2)]
        assert c.read(*got, off2, back) == 0
        want = c.expect_read(off2, back, off2[-1] + 2, out_dtype)
        for a, b in zip(got, want):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("fmt", [I8, I4, FP8])
def test_single_tokens_fill_a_page(fmt):
    c = Cache(2, 2, 64, 16, 3, [fmt], seed=4)
    state = c.host()
    for j in range(35):
        k, v = chunk(2, 2, 64, torch.bfloat16, 100 + j, 1 + j % 7)
        assert c.write(k, v, [0, 1, 2], [j, j + 9]) == 0
        c.expect_write(state, k, v, [0, 1, 2], [j, j + 9])
        c.same(state)


@pytest.mark.parametrize("fmt", [I8, I4, FP8])
def test_zeros_infinities_and_nan(fmt):
    c = Cache(4, 1, 64, 16, 2, [fmt], seed=5)
    state = c.host()
    k, v = chunk(40, 1, 64, torch.float32, 6)
    k[0:10], v[0:10] = 0, 0                                     # a page of zeros gets scale 0
    k[12, 0, 3], v[15, 0, 60] = float("nan"), float("nan")      # left out of max|x|
    k[23, 0, 1] = float("inf")
    v[33, 0] = float("nan")
    off, starts = [0, 10, 20, 30, 40], [0, 0, 6, 3]
    assert c.write(k, v, off, starts) == 0
    with np.errstate(all="ignore"):
        c.expect_write(state, k, v, off, starts)
    c.same(state)


def test_strided_rows_and_rows_behind_the_chunk():
    c = Cache(3, 2, 128, 16, 4, [I8], seed=7)
    state = c.host()
    packed = torch.randn((30, 5, 128), device="cuda").to(torch.bfloat16)
    k, v = packed[:, :2], packed[:, 3:]
    off, starts = [2, 9, 9, 20], [4, 0, 30]                     # rows 0, 1 and 20 .. belong to nobody
    assert c.write(k, v, off, starts) == 0
    c.expect_write(state, k, v, off, starts)
    c.same(state)
    out = torch.full((30, 5, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    assert c.read(out[:, :2], out[:, 3:], off, starts) == 0
    want = c.expect_read(off, starts, 30, torch.bfloat16)
    assert torch.equal(out[:, :2].cpu(), want[0]) and torch.equal(out[:, 3:].cpu(), want[1])
    assert (out[:, 2] == 9).all()


def test_many_sequences():
    B = 700
    lens = [i % 3 for i in range(B)]
    off = [0] + np.cumsum(lens).tolist()
    starts = [(i * 5) % 30 for i in range(B)]
    c = Cache(B, 1, 64, 8, 4, [I4], seed=8)
    state = c.host()
    k, v = chunk(off[-1], 1, 64, torch.bfloat16, 9)
    assert c.write(k, v, off, starts) == 0
    c.expect_write(state, k, v, off, starts)
    c.same(state)
    got = [torch.full((off[-1], 1, 64), 9.0, device="cuda") for _ in range(2)]
    assert c.read(*got, off, starts) == 0
    for a, b in zip(got, c.expect_read(off, starts, off[-1], torch.float32)):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("what,bit", [("slot", binding.DEVERR_PAGE_ID), ("negative", binding.DEVERR_PAGE_ID),
                                      ("format", binding.DEVERR_PAGE_FMT), ("pool", binding.DEVERR_POOL)])
def test_bad_pages_are_skipped_and_reported(what, bit):
    c = Cache(2, 2, 64, 16, 3, [I8, BF16], seed=10)
    state = c.host()
    k, v = chunk(60, 2, 64, torch.bfloat16, 11)
    off, starts = [0, 30, 60], [3, 16]
    if what in ("slot", "negative"):
        c.t_table[0, 1] = 1000 if what == "slot" else -1
    else:
        c.t_fmt[0, 1] = 7 if what == "format" else FP8
    assert c.write(k, v, off, starts) == 0
    assert int(c.err.item()) == bit
    # as if the page did not exist: the tokens around it are written
    c.expect_write(state, k[:13], v[:13], [0, 13, 13], [3, 0])
    c.expect_write(state, k[29:], v[29:], [0, 1, 31], [32, 16])
    c.same(state)
    c.err.zero_()
    got = [torch.full((60, 2, 64), 9.0, device="cuda") for _ in range(2)]
    assert c.read(*got, off, starts) == 0
    assert int(c.err.item()) == bit
    assert (got[0][13:29] == 9).all() and not (got[0][:13] == 9).any() and not (got[0][29:] == 9).any()


@pytest.mark.parametrize("off,starts", [([0, 30, 20], [0, 0]), ([0, 10, 61], [0, 0]), ([-1, 10, 20], [0, 0]),
                                        ([0, 10, 20], [-1, 0]), ([0, 10, 20], [0, 39]), ([5, 3, 20], [0, 0])])
def test_bad_offsets_are_reported_and_nothing_else_is_touched(off, starts):
    c = Cache(2, 1, 64, 16, 3, [I8], seed=12)
    before = c.host()
    k, v = chunk(60, 1, 64, torch.bfloat16, 13)
    assert c.write(k, v, off, starts) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN
    after = c.host()
    for b in range(2):
        n = off[b + 1] - off[b]
        if off[b] < 0 or n < 0 or off[b + 1] > 60 or starts[b] < 0 or starts[b] + n > 48:
            for p in range(3):
                assert np.array_equal(before[0][I8][c.table[b, p]], after[0][I8][c.table[b, p]])
    c.err.zero_()
    got = [torch.full((60, 1, 64), 9.0, device="cuda") for _ in range(2)]
    assert c.read(*got, off, starts) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN


def test_captured_write_and_read():
    c = Cache(2, 2, 128, 16, 8, [I8], seed=14)
    start_k, start_s = c.k[I8].clone(), c.scales[I8].clone()
    k, v = chunk(20, 2, 128, torch.bfloat16, 15)
    off = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    starts = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    out = [torch.zeros_like(k) for _ in range(2)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        assert binding.write_kv(*c.args(), off, starts, k, v, stream=s) == 0
        assert binding.read_kv(*c.args(), off, starts, *out, stream=s) == 0
    for x in (3, 40):                                          # a replay sees what the buffers hold now
        starts[0] = x
        c.k[I8].copy_(start_k)
        c.scales[I8].copy_(start_s)
        state = c.host()
        g.replay()
        torch.cuda.synchronize()
        c.expect_write(state, k, v, [0, 7, 20], [x, 0])
        assert np.array_equal(c.k[I8].cpu().numpy(), state[0][I8])
        want = c.expect_read([0, 7, 20], [x, 0], 20, torch.bfloat16)
        assert torch.equal(out[0].cpu(), want[0]) and torch.equal(out[1].cpu(), want[1])


def test_offsets_beyond_32_bits():
    d, hkv, P = 128, 8, 512
    pages = (1 << 32) // (hkv * P * d) + 5
    kp = torch.zeros((pages, hkv, P, d), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    sc = torch.zeros((pages, hkv, 2), device="cuda")
    pool = binding.pool_struct(hkv, d, P, {I8: kp}, {I8: vp}, {I8: sc})
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0], dtype=torch.int32, device="cuda")
    k, v = chunk(600, hkv, d, torch.bfloat16, 16)
    out = [torch.zeros((600, hkv, d), device="cuda") for _ in range(2)]
    assert binding.write_kv(pool, table, None, I8, off, starts, k, v) == 0
    assert binding.read_kv(pool, table, None, I8, off, starts, *out) == 0
    torch.cuda.synchronize()
    # half a step of the page's scale, max|x| / 127 with |x| below 6
    assert (out[0] - k.float()).abs().max() <= 6 / 127 / 2 * 1.001
    assert kp[pages - 1].any() and not kp[1:pages - 1].any()


def test_offsets_that_fit_several_sequences_stay_inside_the_rows():
    # out of order, so that one block's place fits three sequences, of different lengths: rows of the
    # one that is in order are its own or untouched, and no row from outside the chunk is stored
    c = Cache(4, 1, 64, 8, 8, [I8], seed=22)
    k, v = chunk(60, 1, 64, torch.bfloat16, 23)
    before = c.host()
    assert c.write(k, v, [0, 60, 0, 40, 3], [0, 0, 0, 0]) == 0
    assert int(c.err.item()) == binding.DEVERR_SEQ_LEN
    after = c.host()
    for b in (1, 3):
        for p in range(8):
            assert np.array_equal(before[0][I8][c.table[b, p]], after[0][I8][c.table[b, p]])


@pytest.mark.parametrize("fmt", [I8, I4, FP8])
@pytest.mark.parametrize("top", [1.0, 2.9921875, 0.671875, 2.0 ** -60 * 1.1171875, 2.0 ** -64 * 0.9921875, 2.0 ** 70 * 1.6640625, 2.0 ** -126,
                                 2.0 ** -133, 3.3895314e38, float("inf")])
def test_codes_of_every_bfloat16(fmt, top):
    # every value up to `top`, which sets the scale, signs, zeros, subnormals and NaN among them
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    t = torch.tensor([top]).to(torch.bfloat16)
    every = torch.where(every.abs() > t, t, every)
    x = every.view(512, 1, 128).cuda()
    c = Cache(1, 1, 128, 512, 1, [fmt], seed=24)
    state = c.host()
    assert c.write(x, x.flip(0), [0, 512], [0]) == 0
    with np.errstate(all="ignore"):
        c.expect_write(state, x, x.flip(0), [0, 512], [0])
    c.same(state)


@pytest.mark.parametrize("fmt", [I8, I4, FP8])
@pytest.mark.parametrize("top", [448.0, 1.2345678, 3.1415927e-15, 7.7e12])
def test_codes_beside_the_ties(fmt, top):
    # fp32 values a few units in the last place around every tie's multiple of the scale
    rng = np.random.default_rng(25)
    scale = np.float32(top) / np.float32(QMAX[fmt])
    if fmt == FP8:
        codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        ties = (codes[1:] + codes[:-1]) / 2
    else:
        ties = np.arange(int(QMAX[fmt])) + 0.5
    at = (ties[rng.integers(0, len(ties), 64 * 2 * 128)] * float(scale)).astype(np.float32)
    x = (at.view(np.int32) + rng.integers(-3, 4, at.shape).astype(np.int32)).view(np.float32) * rng.choice([-1, 1], at.shape).astype(np.float32)
    x = np.minimum(np.abs(x), np.float32(top)) * np.sign(x)
    x = torch.from_numpy(x.astype(np.float32)).view(64, 2, 128)
    x[0, :, 0] = top
    k, v = x.cuda(), x.neg().cuda()
    c = Cache(1, 2, 128, 64, 1, [fmt], seed=26)
    state = c.host()
    assert c.write(k, v, [0, 64], [0]) == 0
    c.expect_write(state, k, v, [0, 64], [0])
    c.same(state)


@pytest.mark.parametrize("old", [-5.0, float("nan"), 0.0, 2.0 ** -140])
@pytest.mark.parametrize("fmt", [I8, I4, FP8])
def test_kept_rows_under_scales_that_no_write_leaves(fmt, old):
    c = Cache(1, 2, 64, 16, 1, [fmt], seed=27)
    c.scales[fmt].fill_(old)
    state = c.host()
    k, v = chunk(4, 2, 64, torch.bfloat16, 28)
    assert c.write(k, v, [0, 4], [9]) == 0
    with np.errstate(all="ignore"):
        for w, rows in enumerate((k, v)):       # max(old, max|x| / Q), where a NaN is left out
            for g in range(2):
                x = rows[:, g].float().cpu().numpy()
                scale = np.float32(np.abs(x).max()) / np.float32(QMAX[fmt])
                page = state[w][fmt][int(c.table[0, 0]), g]
                page[:9] = encode(decode_rows(page[:9].copy(), fmt, 64).astype(np.float32) * np.float32(old), fmt, scale)
                page[9:13] = encode(x, fmt, scale)
                state[2][fmt][int(c.table[0, 0]), g, w] = scale
    # (slots that hold no page keep `old`, a NaN among them)
    for w, pool in enumerate((c.k, c.v)):
        assert np.array_equal(pool[fmt].cpu().numpy(), state[w][fmt])
    assert np.array_equal(c.scales[fmt].cpu().numpy(), state[2][fmt], equal_nan=True)
