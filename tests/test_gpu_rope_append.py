"""Norm, rotation and cache write of a step's new tokens (cfr_qk_norm_rope_append)
against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from paged_long_context_b200 import binding, synth

pytestmark = pytest.mark.gpu
F32, BF16 = synth.F32, synth.BF16
TORCH = {F32: torch.float32, BF16: torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from paged_long_context_b200 import build
    build.build()


class Step:
    def __init__(self, T=9, Hq=8, Hkv=2, d=128, P=16, B=3, pages=6, in_fmt=BF16, fmts=(BF16,), rot=None, norm=True,
                 interleaved=False, seed=0, far=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.Hq, self.Hkv, self.d, self.P, self.rot = T, Hq, Hkv, d, P, d if rot is None else rot
        dt = TORCH[in_fmt]
        self.qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g).to(dt).cuda()
        self.q = self.qkv[:, :Hq * d].view(T, Hq, d)
        self.k = self.qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        self.v = self.qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        self.qw = (1 + 0.2 * torch.randn((d,), generator=g)).cuda() if norm else None
        self.kw = (1 + 0.2 * torch.randn((d,), generator=g)).cuda() if norm else None
        cells = rng.permutation(B * pages * P)[:T]
        self.seq = torch.from_numpy((cells // (pages * P)).astype(np.int32)).cuda()
        self.tok = torch.from_numpy((cells % (pages * P)).astype(np.int32)).cuda()
        self.pos = (self.tok + far).to(torch.int32)
        self.inv = (10000.0 ** (-torch.arange(0, self.rot, 2, dtype=torch.float64) / max(self.rot, 1))).cuda() if self.rot else None
        self.interleaved = interleaved
        n = B * pages + 2
        self.kp = {f: torch.randn((n, Hkv, P, d), generator=g).to(TORCH[f]).cuda() for f in fmts}
        self.vp = {f: torch.randn((n, Hkv, P, d), generator=g).to(TORCH[f]).cuda() for f in fmts}
        self.before = {f: (self.kp[f].clone(), self.vp[f].clone()) for f in fmts}
        self.pool = binding.pool_struct(Hkv, d, P, self.kp, self.vp)
        self.table = torch.from_numpy(rng.permutation(n)[:B * pages].reshape(B, pages).astype(np.int32)).cuda()
        self.fmt = rng.choice(list(fmts), size=(B, pages)).astype(np.uint8)
        self.t_fmt = torch.from_numpy(self.fmt).cuda() if len(fmts) > 1 else None
        self.uniform = fmts[0]
        self.q_out = torch.full((T, Hq, d), 5.0, dtype=dt, device="cuda")
        self.err = torch.zeros((1,), dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        return binding.qk_norm_rope_append(
            self.pool, self.q, self.k, self.v, self.pos if self.rot else None, self.inv, self.q_out, self.table, self.t_fmt,
            self.uniform, self.seq, self.tok, q_weight=self.qw, k_weight=self.kw, eps=1e-6, interleaved=self.interleaved,
            err=self.err, stream=stream)

    def turned(self, x, w):
        """(value, sum of the magnitudes that meet in it) in 64 bits."""
        y = x.double().cpu()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double().cpu()
        mag = y.abs().clone()
        h = self.rot // 2
        if h:
            a = self.pos.double().cpu()[:, None] * self.inv.cpu()[None]
            c, s = a.cos()[:, None], a.sin()[:, None]
            i, j = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.interleaved else (slice(0, h), slice(h, self.rot))
            p, q = y[..., i].clone(), y[..., j].clone()
            y[..., i], y[..., j] = p * c - q * s, q * c + p * s
            mag[..., i] = mag[..., j] = p.abs() + q.abs()
        return y, mag

    def check(self, written=None):
        torch.cuda.synchronize()
        # fp32 chain: the norm's sum of d squares (d / 2 roundings of the root), its products, the two products and sum
        # of a rotation and the sines' own error: under 2^-17 of the magnitudes; then half a step of the stored type
        def near(got, want, mag):
            tol = 2.0 ** -17 * mag + torch.finfo(got.dtype).eps / 2 * want.abs() * 1.01
            off = (got.double().cpu() - want).abs()
            assert (off <= tol).all(), (off / tol.clamp(min=1e-30)).max()
        near(self.q_out, *self.turned(self.q, self.qw))
        want_k, mag_k = self.turned(self.k, self.kw)
        want = {f: (a.clone(), b.clone()) for f, (a, b) in self.before.items()}
        for t in range(self.T) if written is None else written:
            b, j = int(self.seq[t]), int(self.tok[t])
            f, slot = int(self.fmt[b, j // self.P]), int(self.table[b, j // self.P])
            near(self.kp[f][slot, :, j % self.P], want_k[t], mag_k[t])
            assert torch.equal(self.vp[f][slot, :, j % self.P], self.v[t].to(TORCH[f]))
            want[f][0][slot, :, j % self.P] = self.kp[f][slot, :, j % self.P]
            want[f][1][slot, :, j % self.P] = self.vp[f][slot, :, j % self.P]
        for f in want:                           # nothing else was written
            assert torch.equal(self.kp[f], want[f][0]) and torch.equal(self.vp[f], want[f][1])


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (128, 0), (64, 64), (64, 48), (64, 32), (128, 112)])
@pytest.mark.parametrize("in_fmt", [BF16, F32], ids=["bf16", "f32"])
def test_norm_and_rotation(in_fmt, d, rot, norm, interleaved):
    s = Step(d=d, rot=rot, norm=norm, interleaved=interleaved, in_fmt=in_fmt, fmts=(in_fmt,))
    assert s.run() == 0
    s.check()
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (32, 8, 1), (5, 1, 33), (20, 4, 7), (64, 8, 3), (32, 32, 5), (256, 2, 2)])
@pytest.mark.parametrize("P", [8, 24, 512])
def test_head_layouts_and_pages(Hq, Hkv, T, P):
    s = Step(T=T, Hq=Hq, Hkv=Hkv, P=P, pages=2 if P == 512 else 6, seed=T)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("in_fmt", [BF16, F32], ids=["bf16", "f32"])
def test_pages_of_both_hot_formats(in_fmt):
    s = Step(T=60, fmts=(BF16, F32), in_fmt=in_fmt, seed=3)
    assert s.run() == 0
    s.check()


def test_far_positions():
    # a position of 2^31 - 1 at frequency 1: its angle is off by 128 rad in 32 bits
    s = Step(T=12, far=2 ** 31 - 200, in_fmt=F32, fmts=(F32,), seed=4)
    assert s.run() == 0
    s.check()


def test_padded_rows_and_bad_places():
    s = Step(T=8, seed=5)
    s.seq[1] = -1
    s.tok[2] = -1
    assert s.run() == 0
    s.check(written=[0, 3, 4, 5, 6, 7])
    assert int(s.err.item()) == 0
    for change, bit in ((lambda: s.seq.__setitem__(3, 3), binding.DEVERR_SEQ_LEN),
                        (lambda: s.tok.__setitem__(4, 96), binding.DEVERR_SEQ_LEN)):
        change()
        s.err.zero_()
        assert s.run() == 0
        torch.cuda.synchronize()
        assert int(s.err.item()) == bit
    s2 = Step(T=1, seed=6)
    s2.table[int(s2.seq[0]), int(s2.tok[0]) // 16] = 99
    assert s2.run() == 0
    s2.check(written=[])
    assert int(s2.err.item()) == binding.DEVERR_PAGE_ID
    s3 = Step(T=1, seed=6, fmts=(BF16, F32))
    s3.t_fmt[int(s3.seq[0]), int(s3.tok[0]) // 16] = synth.I8
    assert s3.run() == 0
    s3.check(written=[])
    assert int(s3.err.item()) == binding.DEVERR_PAGE_FMT


def test_non_finite_rows_stay_in_their_rows():
    s = Step(T=4, seed=7)
    s.q[1, 2, 5] = float("nan")
    s.k[2, 0, 3] = float("inf")
    assert s.run() == 0
    torch.cuda.synchronize()
    bad = ~torch.isfinite(s.q_out)
    assert bad[1, 2].any()
    bad[1, 2] = False
    assert not bad.any()


def test_captured_step_sees_new_positions():
    s = Step(T=5, seed=8)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        assert s.run(stream=st) == 0
    s.pos += 1000
    g.replay()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("T,interleaved,in_fmt", [(4096, False, BF16), (4099, True, BF16), (5001, False, F32)])
def test_long_steps(T, interleaved, in_fmt):
    # enough tokens for a block to take several of them, and a last block that is not full
    s = Step(T=T, Hq=3, Hkv=1, B=4, pages=80, in_fmt=in_fmt, fmts=(in_fmt,), interleaved=interleaved, seed=9, far=70000)
    s.seq[5], s.tok[T - 1] = -1, -1
    assert s.run() == 0
    s.check(written=[t for t in range(T) if t not in (5, T - 1)])
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("far", [0, 130000, 1000000])
def test_sines_and_cosines(far, interleaved):
    # rows of ones against zeros come back as the cosines and sines themselves: each within the functions' one unit in
    # the last place (2^-24 at most) and the rounding of an angle of an eighth of a turn (2^-28 of a turn)
    s = Step(T=1500, Hq=2, Hkv=1, d=128, P=512, B=1, pages=4, in_fmt=F32, fmts=(F32,), norm=False, interleaved=interleaved, far=far)
    i, j = (slice(0, 128, 2), slice(1, 128, 2)) if interleaved else (slice(0, 64), slice(64, 128))
    s.q[..., i], s.q[..., j] = 1.0, 0.0
    assert s.run() == 0
    torch.cuda.synchronize()
    a = (s.pos.double().cpu()[:, None] * s.inv.cpu()[None])[:, None]
    got = s.q_out.double().cpu()
    tol = 2.0 ** -24 + 2 * np.pi * 2.0 ** -28 + 1e-9
    assert (got[..., i] - a.cos()).abs().max() <= tol
    assert (got[..., j] - a.sin()).abs().max() <= tol
