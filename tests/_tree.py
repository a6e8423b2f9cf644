"""Tree attention in 64 bits from host bytes, with the error bounds of the kernels."""
import numpy as np
import torch

from paged_long_context_b200 import binding, synth
from tests._hostkv import host_kv, host_q, kv_head_of, sigma_of

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24   # half a step, relative: torch.finfo(t).eps / 2


def chain(Q):
    return [(1 << (i + 1)) - 1 for i in range(Q)], list(range(Q))


def random_tree(Q, rng):
    """Ancestor bits and depths of a random tree of Q nodes."""
    masks, depths = [], []
    for i in range(Q):
        parent = int(rng.integers(-1, i)) if i else -1
        masks.append((masks[parent] if parent >= 0 else 0) | (1 << i))
        depths.append(depths[parent] + 1 if parent >= 0 else 0)
    return masks, depths


def as_int64(masks, device="cuda"):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks],
                        dtype=torch.int64, device=device)


class TreeCall:
    """One call on a synthetic case (spec.num_queries drafts a sequence)."""

    def __init__(self, case, masks=None, depths=None, q_lens=None, cap=0.0, out_dtype=torch.bfloat16):
        self.case, self.masks, self.depths, self.q_lens, self.cap = case, masks, depths, q_lens, cap
        dev, B, Q, H, d = case.device, case.batch, case.num_queries, case.num_q_heads, case.head_dim
        dt = torch.float32 if case.q_fmt == synth.F32 else torch.bfloat16
        self.q = case.q.view(dt).view(B, Q, H, d)
        self.out = torch.full((B, Q, H, d), 7.0, dtype=out_dtype, device=dev)
        self.lse = torch.full((B, Q, H), 7.0, dtype=torch.float32, device=dev)
        self.err = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.pool = binding.kv_pool_struct(case)
        n = binding.tree_workspace_size(B, Q, H, case.num_kv_heads, d)
        assert n > 0
        self.workspace = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.t_mask = None if masks is None else as_int64(masks, dev)
        self.t_depths, self.t_q_lens = i32(depths), i32(q_lens)

    def run(self, stream=None):
        c = self.case
        hm = None if c.head_map is None else c.head_map.cpu()
        return binding.paged_decode_tree(
            self.pool, self.q, c.page_table, c.seq_lens, self.out, self.lse, self.workspace,
            page_fmt=c.page_fmt, uniform_fmt=c.uniform_fmt, q_lens=self.t_q_lens, tree_mask=self.t_mask,
            depths=self.t_depths, head_map=hm, alibi_slopes=c.alibi_slopes, softmax_scale=c.softmax_scale,
            logit_cap=self.cap, err=self.err, stream=stream)

    def reference(self, dropped=()):
        """{(b, i, h): (out, lse, tolerance of out, tolerance of lse)}; `dropped`: tokens (b, j) left out.

        Tolerances, in units of A = sum_j p_j |v_j| (p the exact softmax):
          scores   e = (d + 4) 2^-24 sigma max_j sum |q||k|, and 2^-21 cap where they are capped;
                   2^-23 of the ALiBi term; each p is off by 2 e relative
          sums     (n + 8) 2^-24
          p as an operand  one rounding to 16 bits (bf16): 2^-8, none where everything is fp32
          out      half a step of its type
        """
        c = self.case.to("cpu")
        Q, d, sig = c.num_queries, c.head_dim, sigma_of(c)
        q = host_q(c).reshape(c.batch, Q, c.num_q_heads, d)
        slopes = None if c.alibi_slopes is None else c.alibi_slopes.double().numpy()
        fp32 = c.q_fmt == synth.F32 or synth.F32 in c.k_pool
        half = F32_HALF if self.out.dtype == torch.float32 else BF16_HALF
        ref = {}
        for b in range(c.batch):
            n, cb = int(c.seq_lens[b]), Q if self.q_lens is None else self.q_lens[b]
            pre = n - cb
            if cb == 0:
                continue
            masks = chain(Q)[0] if self.masks is None else self.masks[b]
            depth = np.array(range(Q) if self.depths is None else self.depths[b])
            pos = np.arange(n)
            pos[pre:] = pre + depth[:cb]
            kv = {}
            for h in range(c.num_q_heads):
                g = kv_head_of(c, h)
                if g not in kv:
                    kv[g] = host_kv(c, b, g)
                K, V = kv[g]
                for i in range(cb):
                    seen = np.ones(n, bool)
                    for k in range(cb):
                        seen[pre + k] = bool((masks[i] >> k) & 1)
                    for bb, j in dropped:
                        if bb == b:
                            seen[j] = False
                    if not seen.any():
                        ref[b, i, h] = (np.zeros(d), -np.inf, np.zeros(d), 0.0)
                        continue
                    Ks, Vs, ps = K[seen], V[seen], pos[seen]
                    s = Ks @ q[b, i, h] * sig
                    e = (d + 4) * F32_HALF * sig * float((np.abs(Ks) @ np.abs(q[b, i, h])).max())
                    if self.cap:
                        s = self.cap * np.tanh(s / self.cap)
                        e += 2.0 ** -21 * self.cap
                    if slopes is not None:
                        s = s - slopes[h] * (pre + depth[i] - ps)
                        near = s >= s.max() - 30        # tokens further below carry no weight
                        e += 2.0 ** -22 * float(np.abs(slopes[h] * (pre + depth[i] - ps))[near].max())
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    o = p @ Vs / l
                    A = p @ np.abs(Vs) / l
                    rel = 2 * e + (len(s) + 8) * F32_HALF + 2.0 ** -20 + (0.0 if fp32 else BF16_HALF)
                    lse = m + np.log(l)
                    ref[b, i, h] = (o, lse, rel * A + half * np.abs(o) * 1.01,
                                    2 * e + (len(s) + 8) * F32_HALF + 2.0 ** -20 * max(1.0, abs(lse)))
        return ref

    def check(self, dropped=(), skip=()):
        torch.cuda.synchronize()
        out, lse = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        ref = self.reference(dropped)
        for b in range(self.case.batch):
            for i in range(self.case.num_queries):
                for h in range(self.case.num_q_heads):
                    if (b, i, h) in skip:
                        continue
                    if (b, i, h) not in ref:       # a row behind the sequence's drafts
                        assert (out[b, i, h] == 7.0).all() and lse[b, i, h] == 7.0, (b, i, h)
                        continue
                    o, l, to, tl = ref[b, i, h]
                    off = np.abs(out[b, i, h] - o)
                    assert (off <= to).all(), f"{(b, i, h)}: off by {off.max()}, {(off / np.maximum(to, 1e-30)).max():.2f} of tolerance"
                    if np.isneginf(l):
                        assert np.isneginf(lse[b, i, h])
                    else:
                        assert abs(lse[b, i, h] - l) <= tl, f"{(b, i, h)}: lse {lse[b, i, h]} for {l}"


def tree_case(lens, Q, Hq=8, Hkv=2, d=128, P=16, fmt="bf16", q_fmt="bf16", alibi=False, seed=3, **kw):
    spec = synth.CaseSpec("tree", len(lens), Hq, Hkv, d, P, seq_lens=list(lens), fmt=fmt, q_fmt=q_fmt,
                          alibi=alibi, num_queries=Q, spare_pages=2, **kw)
    return synth.make_case(spec, seed, "cuda")
