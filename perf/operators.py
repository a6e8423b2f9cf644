"""Cases for measuring the cache-writing and tree-verification operators.

Four operators that a speculative decoder over a paged cache runs next to the
decode itself:

  rope   norms of queries and keys for each head, their position rotation and
         the write of K and V into the hot tier's pages, in one pass
  write  a ragged chunk of new tokens stored into (quantised) pages as it
         arrives, and the touched pages read back
  read   cached tokens read back as dense rows, dequantised
  tree   attention of a tree of drafted tokens over the paged cache, optionally
         with ALiBi and with scores capped by a tanh

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it makes the calls of the library's entry points.
Pools, page tables and formats are laid out as include/cfr_paged.h describes.
"""
import math

import torch

own = False

F32, BF16, I8, I4, FP8 = 0, 1, 2, 3, 4
FMT = {"f32": F32, "bf16": BF16, "i8": I8, "i4": I4, "fp8": FP8}
QMAX = {I8: 127.0, I4: 7.0, FP8: 448.0}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
THETA = 500000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence: the latency of a single decode step
        dict(name="rope_step", op="rope", batch=1, lo=1, hi=1, far=20000, ahead=0, hq=32, hkv=8, d=128, rot=128,
             page=16, fmt="bf16", pairs="half", norm=True),
        # prefill chunks of a ragged batch going into 16-token pages
        dict(name="rope_prompt", op="rope", batch=8, lo=257, hi=4096, far=6000, ahead=0, hq=32, hkv=8, d=128, rot=128,
             page=16, fmt="bf16", pairs="half", norm=True),
        # fp32 cache, 32 heads of 64, half of each head rotated in neighbouring pairs, far positions
        dict(name="rope_f32_partial", op="rope", batch=3, lo=85, hi=1001, far=3001, ahead=1000000, hq=32, hkv=32, d=64, rot=32,
             page=512, fmt="f32", pairs="neighbours", norm=False),
        # one token a sequence appended into int8 pages that are part full
        dict(name="write_step_i8", op="write", batch=16, lo=1, hi=1, far=4000, hkv=8, d=128, page=16, fmt="i8",
             new="bf16", out="bf16"),
        # ragged prompt chunks going straight into the coldest tier
        dict(name="write_prompt_i4", op="write", batch=8, lo=300, hi=8192, far=9000, hkv=8, d=128, page=256,
             fmt="i4", new="bf16", out="bf16"),
        # E4M3 pages of 16 tokens, heads of 64, rows that arrive in 32 bits
        dict(name="write_fp8_d64", op="write", batch=5, lo=33, hi=2500, far=700, hkv=8, d=64, page=16, fmt="fp8",
             new="f32", out="bf16"),
        # a cached prefix of every sequence brought back for a dense prefill
        dict(name="read_tiered", op="read", batch=8, lo=9001, hi=32768, hkv=8, d=128, page=256, fmt="tiered",
             out="bf16"),
        # a few hundred int8 tokens of one sequence
        dict(name="read_i8_small", op="read", batch=1, lo=333, hi=333, hkv=8, d=64, page=16, fmt="i8", out="f32"),
        # a short chat turn: seven drafted tokens of one sequence
        dict(name="tree_small", op="tree", batch=1, lo=1013, hi=1013, nq=7, ragged=False, hq=32, hkv=8, d=128,
             page=16, fmt="bf16", cap=0.0, alibi=False),
        # the ragged serving batch, up to 64 drafted tokens a sequence
        dict(name="tree_wide", op="tree", batch=16, lo=1024, hi=32768, nq=64, ragged=True, hq=32, hkv=8, d=128,
             page=16, fmt="bf16", cap=0.0, alibi=False),
        # int4 / int8 / bf16 tiers of long sequences, capped scores, 16 drafted tokens
        dict(name="tree_tiered_cap", op="tree", batch=8, lo=32768, hi=32768, nq=16, ragged=False, hq=32, hkv=8,
             d=128, page=256, fmt="tiered", cap=50.0, alibi=False),
        # one sequence of a million tokens with ALiBi, eight drafted tokens
        dict(name="tree_long", op="tree", batch=1, lo=1048576, hi=1048576, nq=8, ragged=False, hq=64, hkv=8, d=128,
             page=512, fmt="bf16", cap=0.0, alibi=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree"])
    if op == "rope":
        hq, hkv = rng.choice([(32, 8), (32, 32), (8, 1), (20, 4), (64, 8)])
        d = rng.choice([64, 128])
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, max(1, 16000 // batch))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.randint(1, 8)), hi=hi, far=_log_int(rng, 1, 9000),
                    ahead=rng.choice([0, 0, 131072, 1000000]), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, 16]), page=rng.choice([8, 16, 24, 64, 256, 512]),
                    fmt=rng.choice(["bf16", "bf16", "f32"]), pairs=rng.choice(["half", "neighbours"]),
                    norm=rng.random() < 0.7)
    if op == "write":
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, max(1, 32000 // batch))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.randint(1, 8)), hi=hi, far=_log_int(rng, 1, 9000),
                    hkv=rng.choice([1, 2, 8, 8, 32]) if hi * batch < 8000 else rng.choice([1, 2, 8]),
                    d=rng.choice([64, 128, 128]), page=rng.choice([8, 16, 24, 64, 256, 512]),
                    fmt=rng.choice(["i8", "i4", "fp8", "bf16"]), new=rng.choice(["bf16", "bf16", "f32"]), out="bf16")
    if op == "read":
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, max(1, 200000 // batch))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.randint(1, 8)), hi=hi, hkv=rng.choice([1, 2, 8]),
                    d=rng.choice([64, 128, 128]), page=rng.choice([8, 16, 24, 64, 256, 512]),
                    fmt=rng.choice(["i8", "i4", "fp8", "bf16", "tiered"]), out=rng.choice(["bf16", "bf16", "f32"]))
    batch = _log_int(rng, 1, 32)
    hq, hkv = rng.choice([(32, 8), (32, 8), (64, 8), (8, 1), (20, 4), (16, 16)])
    nq = _log_int(rng, 1, 64)
    most = min(300000, 500000000 // (hq * nq))  # tokens of the whole batch
    hi = max(nq + 1, _log_int(rng, 64, max(65, most // batch)))
    return dict(op=op, batch=batch, lo=max(nq, hi // rng.randint(1, 16)), hi=hi, nq=nq, ragged=rng.random() < 0.5,
                hq=hq, hkv=hkv, d=rng.choice([64, 128, 128]), page=rng.choice([16, 16, 32, 64, 128, 256, 512]),
                fmt=rng.choice(["bf16", "bf16", "i8", "i4", "fp8", "tiered"]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                alibi=rng.random() < 0.3)


def _spread(case):
    """Lengths of the batch's sequences: from lo to hi, the odd ones among them."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    return [max(lo, lo + (hi - lo) * i // (n - 1) - (i * 7 % 5 if i < n - 1 else 0)) for i in range(n)]


def _drafts(case):
    """Drafted tokens of each sequence (a ragged batch verifies trees of unequal size)."""
    nq = case["nq"]
    return [nq - (i * 5 % (nq // 2 + 1) if case["ragged"] else 0) for i in range(case["batch"])]


def _row_bytes(fmt, d):
    return {F32: 4 * d, BF16: 2 * d, I8: d, I4: d // 2, FP8: d}[fmt]


def _tier(case, lens):
    """Format of every page of every sequence: uniform, or oldest quarter int4, next half int8, newest quarter bf16."""
    out = []
    for n in lens:
        pages = -(-n // case["page"])
        if case["fmt"] == "tiered":
            hot, warm = -(-pages // 4), pages // 2
            out.append([I4] * (pages - hot - warm) + [I8] * warm + [BF16] * hot)
        else:
            out.append([FMT[case["fmt"]]] * pages)
    return out


def _cache_bytes(case, lens):
    """Bytes of K and V of the first lens[b] tokens of every sequence, scales among them."""
    total, P, h, d = 0, case["page"], case["hkv"], case["d"]
    for n, fmts in zip(lens, _tier(case, lens)):
        for i, f in enumerate(fmts):
            total += 2 * h * (min(P, n - i * P) * _row_bytes(f, d) + (4 if f in QMAX else 0))
    return total


def work(case):
    d, op = case["d"], case["op"]
    lens = _spread(case)
    T = sum(lens)
    if op == "rope":
        e = 4 if case["fmt"] == "f32" else 2
        values = T * d * (case["hq"] + 2 * case["hkv"])
        return dict(bytes=2 * e * values + T * 12, flops=T * (case["hq"] + case["hkv"]) * (4 * d + 3 * case["rot"]))
    if op == "write":
        e = 4 if case["new"] == "f32" else 2
        back = sum(n + s % case["page"] for n, s in zip(lens, _starts(case)))
        kept = _cache_bytes(dict(case), [s % case["page"] for s in _starts(case)])
        return dict(bytes=2 * T * case["hkv"] * d * e + 2 * _cache_bytes(case, lens) + kept
                    + 2 * back * case["hkv"] * d * (4 if case["out"] == "f32" else 2),
                    flops=6 * T * case["hkv"] * d)
    if op == "read":
        e = 4 if case["out"] == "f32" else 2
        return dict(bytes=_cache_bytes(case, lens) + 2 * T * case["hkv"] * d * e, flops=2 * T * case["hkv"] * d)
    rows = [c * case["hq"] for c in _drafts(case)]
    return dict(bytes=_cache_bytes(case, lens) + sum(rows) * (4 * d + 4) + sum(_drafts(case)) * 8,
                flops=sum(4 * d * r * n for r, n in zip(rows, lens)))


def _starts(case):
    """Tokens that each sequence holds before a chunk is written (0 to `far`, most of them inside a page)."""
    return [(case["far"] * (i + 1) // case["batch"]) - (i * 3 % 4 if case["far"] > 8 else 0) for i in range(case["batch"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _encode(x, scale, fmt):
    """Codes (as fp32 values) of x, given its scale: round to nearest even of the fp32 quotient."""
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    if fmt == FP8:
        return q.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return torch.round(q).clamp(-QMAX[fmt], QMAX[fmt])


def _pack(codes, fmt):
    """Stored bytes (uint8, last axis) of code values."""
    if fmt == FP8:
        return codes.to(torch.float8_e4m3fn).view(torch.uint8)
    if fmt == I8:
        return codes.to(torch.int8).view(torch.uint8)
    n = codes.to(torch.int32) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def _unpack(raw, fmt):
    """Stored bytes -> fp32 values before scaling."""
    if fmt == F32:
        return raw.view(torch.float32)
    if fmt == BF16:
        return raw.view(torch.bfloat16).float()
    if fmt == FP8:
        return raw.view(torch.float8_e4m3fn).float()
    if fmt == I8:
        return raw.view(torch.int8).float()
    lo, hi = (raw & 15).to(torch.int8), (raw >> 4).to(torch.int8)
    both = torch.stack((lo, hi), -1).flatten(-2)
    return torch.where(both > 7, both - 16, both).float()


def _make_pool(gen, slots, hkv, page, d, fmt):
    """One pool of `slots` pages of N(0, 1) rows: (bytes, per-page per-head scales or None)."""
    shape = (slots, hkv, page, d)
    if fmt == F32:
        return torch.randn(shape, device="cuda", generator=gen).view(torch.uint8), None
    if fmt == BF16:
        return torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=gen).view(torch.uint8), None
    raw = torch.empty((slots, hkv, page, _row_bytes(fmt, d)), device="cuda", dtype=torch.uint8)
    scale = torch.empty((slots, hkv), device="cuda")
    step = max(1, (1 << 27) // (hkv * page * d))
    for i in range(0, slots, step):
        x = torch.randn((min(step, slots - i),) + shape[1:], device="cuda", generator=gen)
        scale[i:i + step] = x.abs().amax((2, 3)) / QMAX[fmt]
        raw[i:i + step] = _pack(_encode(x, scale[i:i + step, :, None, None], fmt), fmt)
    return raw, scale


def _make_cache(case, lens, gen, seed):
    """Pools, page table and formats of a cache that has room for lens[b] tokens of every sequence."""
    import random as _random
    rng = _random.Random(seed)
    tiers = _tier(case, lens)
    most = max(len(t) for t in tiers)
    need = {f: sum(t.count(f) for t in tiers) for f in (F32, BF16, I8, I4, FP8)}
    ids = {f: rng.sample(range(n + 3), n + 3) for f, n in need.items() if n}
    table, fmts = [], []
    for t in tiers:
        table.append([ids[f].pop() for f in t] + [0] * (most - len(t)))
        fmts.append(t + [t[-1] if t else BF16] * (most - len(t)))
    s = dict(hkv=case["hkv"], d=case["d"], page=case["page"], max_pages=most, table=_i32(table), k={}, v={}, scales={})
    for f, n in need.items():
        if n:
            s["k"][f], ks = _make_pool(gen, n + 3, case["hkv"], case["page"], case["d"], f)
            s["v"][f], vs = _make_pool(gen, n + 3, case["hkv"], case["page"], case["d"], f)
            if ks is not None:
                s["scales"][f] = torch.stack((ks, vs), -1).contiguous()
    s["kv"] = (s["k"], s["v"])
    s["mixed"] = case["fmt"] == "tiered"
    s["page_fmt"] = torch.tensor(fmts, dtype=torch.uint8).cuda() if s["mixed"] else None
    s["fmt"] = BF16 if s["mixed"] else FMT[case["fmt"]]
    return s


def _ragged(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _spread(case)
    shift = seed % case["batch"]
    lens = lens[shift:] + lens[:shift]  # the same lengths in another order
    op, d, hkv, batch = case["op"], case["d"], case["hkv"], case["batch"]
    off = _ragged(lens)
    T = off[-1]
    seqs = [b for b, n in enumerate(lens) for _ in range(n)]
    if op in ("rope", "write"):
        starts = _starts(case)
        starts = starts[shift:] + starts[:shift]
        s = _make_cache(case, [a + n for a, n in zip(starts, lens)], gen, seed)
        at = [a + i for a, n in zip(starts, lens) for i in range(n)]
    if op == "rope":
        dt = DTYPE[case["fmt"]]
        hq = case["hq"]
        # the packed output of a fused projection: q, k and v are views of it; a few channels are far larger
        qkv = torch.randn((T, (hq + 2 * hkv) * d), device="cuda", generator=gen)
        qkv = (qkv * (1 + 9 * (torch.rand((qkv.shape[1],), device="cuda", generator=gen) < 0.02))).to(dt)
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["new_k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["new_v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        s["seq_ids"], s["token_ids"] = _i32(seqs), _i32(at)
        s["rope_pos"] = s["token_ids"] + case["ahead"]
        s["inv_freq"] = (THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).cuda()
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = 1 + 0.1 * torch.randn((d,), device="cuda", generator=gen)
            s["kw"] = 1 + 0.1 * torch.randn((d,), device="cuda", generator=gen)
        s["neighbours"] = case["pairs"] == "neighbours"
        s["q_out"] = torch.zeros((T, hq, d), device="cuda", dtype=dt)
    elif op == "write":
        dt, P = DTYPE[case["new"]], case["page"]
        s["new_k"] = torch.randn((T, hkv, d), device="cuda", generator=gen).to(dt)
        s["new_v"] = torch.randn((T, hkv, d), device="cuda", generator=gen).to(dt)
        s["seq_ids"], s["token_ids"] = _i32(seqs).long(), _i32(at).long()
        s["off"], s["starts"] = _i32(off), _i32(starts)
        first = [a - a % P for a in starts]  # what is read back: the touched pages up to the chunk's end
        back = [a + n - f for a, n, f in zip(starts, lens, first)]
        s["back_off"], s["back_starts"] = _i32(_ragged(back)), _i32(first)
        s["back_seq"] = _i32([b for b, n in enumerate(back) for _ in range(n)]).long()
        s["back_tok"] = _i32([f + i for f, n in zip(first, back) for i in range(n)]).long()
        s["k_out"] = torch.zeros((sum(back), hkv, d), device="cuda", dtype=DTYPE[case["out"]])
        s["v_out"] = torch.zeros_like(s["k_out"])
    elif op == "read":
        s = _make_cache(case, lens, gen, seed)
        s["off"], s["starts"] = _i32(off), _i32([0] * batch)
        s["back_off"], s["back_starts"] = s["off"], s["starts"]
        s["back_seq"] = _i32(seqs).long()
        s["back_tok"] = _i32([i for n in lens for i in range(n)]).long()
        s["k_out"] = torch.zeros((T, hkv, d), device="cuda", dtype=DTYPE[case["out"]])
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        s = _make_cache(case, lens, gen, seed)
        nq, hq = case["nq"], case["hq"]
        drafts = _drafts(case)
        drafts = drafts[shift:] + drafts[:shift]
        mask, depth = _trees(drafts, nq, seed)
        s["q"] = torch.randn((batch, nq, hq, d), device="cuda", generator=gen).to(torch.bfloat16)
        s["lens"], s["drafts"] = _i32(lens), _i32(drafts)
        s["mask"] = torch.tensor(mask, dtype=torch.int64).cuda()
        s["depth"] = _i32(depth)
        s["cap"] = case["cap"]
        s["slopes"] = None
        if case["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8 * (i + 1) / hq) for i in range(hq)]).cuda()
        s["out"] = torch.zeros((batch, nq, hq, d), device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros((batch, nq, hq), device="cuda")
        # the scratch that a user's program allocates once for the shapes it serves
        s["workspace"] = None
    s["op"] = op
    return s


def _trees(drafts, nq, seed):
    """A random tree over every sequence's drafted tokens: ancestor bits (itself among them) and depths."""
    import random as _random
    rng = _random.Random(seed + 1)
    masks, depths = [], []
    for n in drafts:
        m, dep = [], []
        for i in range(nq):
            parent = rng.randint(max(-1, i - 8), i - 1)
            m.append((m[parent] if parent >= 0 else 0) | (1 << i))
            dep.append(dep[parent] + 1 if parent >= 0 else 0)
        masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        depths.append(dep)
    return masks, depths


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"rope": _rope, "write": _write, "read": _read, "tree": _tree}[s["op"]](s)


def _values(s, which):
    """Every page of the cache in fp32, the pools of all formats one after another."""
    return torch.cat([_unpack(raw, f) * s["scales"][f][:, :, which, None, None] if f in s["scales"] else _unpack(raw, f)
                      for f, raw in s["kv"[which]].items()])


def _pages(s):
    """Place of every logical page in _values()."""
    if not s["mixed"]:
        return s["table"].long()
    counts = torch.tensor([s["k"][f].shape[0] if f in s["k"] else 0 for f in range(5)], device=s["table"].device)
    base = torch.zeros(5, dtype=torch.int64, device=s["table"].device)
    at = torch.tensor(list(s["k"]), device=s["table"].device)
    base[at] = counts[at].cumsum(0) - counts[at]
    return s["table"].long() + base[s["page_fmt"].long()]


def _check(status):
    if status != 0:
        raise RuntimeError("the call was rejected with status %d" % status)


def _handle(s):
    """The pool description that a user's program keeps with its cache."""
    from paged_long_context_b200 import binding
    if "pool" not in s:
        s["pool"] = binding.pool_struct(s["hkv"], s["d"], s["page"], s["k"], s["v"], s["scales"])
    return binding, s["pool"]


def _rope(s):
    if own:
        binding, pool = _handle(s)
        _check(binding.qk_norm_rope_append(
            pool, s["q"], s["new_k"], s["new_v"], s["rope_pos"], s["inv_freq"], s["q_out"], s["table"], s["page_fmt"],
            s["fmt"], s["seq_ids"], s["token_ids"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
            interleaved=s["neighbours"]))
        return dict(q=s["q_out"], k=_stored(s, "k"), v=_stored(s, "v"))
    ang = s["rope_pos"].double()[:, None] * s["inv_freq"]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    rot = 2 * cos.shape[-1]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["neighbours"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        p, q = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((p, q), -1).flatten(-2) if s["neighbours"] else torch.cat((p, q), -1)
        return torch.cat((r, x[..., rot:]), -1)

    dt = s["q"].dtype
    s["q_out"].copy_(one(s["q"], s["qw"]))
    tok = s["token_ids"].long()
    slot = s["table"].long()[s["seq_ids"].long(), tok // s["page"]]
    _stored(s, "k")[slot, :, tok % s["page"]] = one(s["new_k"], s["kw"]).to(dt)
    _stored(s, "v")[slot, :, tok % s["page"]] = s["new_v"]
    return dict(q=s["q_out"], k=_stored(s, "k"), v=_stored(s, "v"))


def _stored(s, which):
    """The pool of an unquantised cache as values."""
    return s[which][s["fmt"]].view(torch.float32 if s["fmt"] == F32 else torch.bfloat16)


def _write(s):
    fmt, P = s["fmt"], s["page"]
    if own:
        binding, pool = _handle(s)
        _check(binding.write_kv(pool, s["table"], s["page_fmt"], fmt, s["off"], s["starts"], s["new_k"], s["new_v"]))
        _check(binding.read_kv(pool, s["table"], s["page_fmt"], fmt, s["back_off"], s["back_starts"], s["k_out"],
                               s["v_out"]))
    else:
        # each touched page of a sequence, and whether tokens that it already holds stay in it
        seq, tok = s["seq_ids"], s["token_ids"]
        slot = s["table"].long()[seq, tok // P]
        for which, x in (("k", s["new_k"]), ("v", s["new_v"])):
            x, raw, n = x.float(), s[which][fmt], 0 if which == "k" else 1
            if fmt in QMAX:
                old = s["scales"][fmt][:, :, n]
                amax = torch.zeros_like(old).index_reduce_(0, slot, x.abs().amax(-1), "amax")
                first = torch.full((old.shape[0],), P, device=old.device).index_reduce_(0, slot, tok % P, "amin")
                kept = (first > 0) & (first < P)
                new = torch.where((first < P)[:, None],
                                  torch.maximum(amax / torch.full_like(amax, QMAX[fmt]), torch.where(kept[:, None], old, 0 * old)), old)
                stay = torch.nonzero(kept).flatten()
                held = _unpack(raw[stay], fmt) * old[stay][:, :, None, None]
                again = _pack(_encode(held, new[stay][:, :, None, None], fmt), fmt)
                rows = torch.arange(P, device=old.device)[None, None, :, None] < first[stay][:, None, None, None]
                moved = rows & (new[stay] > old[stay])[:, :, None, None]
                raw[stay] = torch.where(moved, again, raw[stay])
                s["scales"][fmt][:, :, n] = new
                raw[slot, :, tok % P] = _pack(_encode(x, new[slot][:, :, None], fmt), fmt)
            else:
                raw[slot, :, tok % P] = (x if fmt == F32 else x.to(torch.bfloat16)).view(torch.uint8)
        _dense(s)
    out = dict(k=s["k_out"], v=s["v_out"])
    if fmt in QMAX:
        out["scales"] = s["scales"][fmt]
    return out


def _dense(s):
    place = _pages(s)[s["back_seq"], s["back_tok"] // s["page"]]
    row = s["back_tok"] % s["page"]
    s["k_out"].copy_(_values(s, 0)[place, :, row])
    s["v_out"].copy_(_values(s, 1)[place, :, row])


def _read(s):
    if own:
        binding, pool = _handle(s)
        _check(binding.read_kv(pool, s["table"], s["page_fmt"], s["fmt"], s["back_off"], s["back_starts"], s["k_out"],
                               s["v_out"]))
    else:
        _dense(s)
    return dict(k=s["k_out"], v=s["v_out"])


def _tree(s):
    q = s["q"]
    batch, nq, hq, d = q.shape
    if own:
        binding, pool = _handle(s)
        if s["workspace"] is None:
            n = binding.tree_workspace_size(batch, nq, hq, s["hkv"], d)
            s["workspace"] = torch.empty((n,), dtype=torch.uint8, device=q.device)
        _check(binding.paged_decode_tree(
            pool, q, s["table"], s["lens"], s["out"], s["lse"], s["workspace"], page_fmt=s["page_fmt"],
            uniform_fmt=s["fmt"], q_lens=s["drafts"], tree_mask=s["mask"], depths=s["depth"], alibi_slopes=s["slopes"],
            logit_cap=s["cap"]))
        return dict(out=s["out"], lse=s["lse"])
    hkv, P, n = s["hkv"], s["page"], s["table"].shape[1] * s["page"]
    place = _pages(s)

    def dense(which):  # [batch, kv head, token, d]
        return _values(s, which)[place].transpose(1, 2).reshape(batch, hkv, n, d)

    # rows of one kv head: (draft, query head of the group)
    rows = q.float().view(batch, nq, hkv, hq // hkv, d).transpose(1, 2).reshape(batch, hkv, -1, d)
    x = (rows @ dense(0).transpose(2, 3)) / math.sqrt(d)
    x = x.view(batch, hkv, nq, hq // hkv, n)
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    j = torch.arange(n, device=q.device)[None]
    first = (s["lens"] - s["drafts"])[:, None].long()
    k = (j - first).clamp(0, 63)  # drafted token that a cache token is
    if s["slopes"] is not None:
        at = torch.where(j < first, j, first + s["depth"].long().gather(1, k.clamp(max=nq - 1)))
        far = (first + s["depth"])[:, :, None] - at[:, None]
        x = x - s["slopes"].view(1, hkv, 1, -1, 1) * far[:, None, :, None].float()
    bit = (s["mask"][:, :, None] >> k[:, None]) & 1
    seen = ((j < first)[:, None] | ((bit == 1) & (j < s["lens"][:, None])[:, None]))[:, None, :, None]
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    live = (j < s["lens"][:, None])[:, None, :, None]
    y = (x / total).view(batch, hkv, -1, n) @ torch.where(live, dense(1), 0.0)
    y = y.view(batch, hkv, nq, hq // hkv, d).transpose(1, 2).reshape(batch, nq, hq, d)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(batch, nq, hq)
    real = (torch.arange(nq, device=q.device)[None] < s["drafts"][:, None])[:, :, None]
    s["out"].copy_(torch.where(real[..., None], y, s["out"].float()))
    s["lse"].copy_(torch.where(real, lse, s["lse"]))
    return dict(out=s["out"], lse=s["lse"])


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _stored64(s, b, lo, hi, which):
    """Tokens [lo, hi) of sequence b as the cache holds them, [token, kv head, d] in 64 bits, page by page."""
    P, parts = s["page"], []
    table = s["table"][b].tolist()
    fmts = s["page_fmt"][b].tolist() if s["mixed"] else [s["fmt"]] * len(table)
    pages = list(range(lo // P, -(-hi // P)))
    at = 0
    while at < len(pages):  # runs of pages of one format
        end = at
        while end < len(pages) and fmts[pages[end]] == fmts[pages[at]]:
            end += 1
        f = fmts[pages[at]]
        ids = torch.tensor([table[p] for p in pages[at:end]], device="cuda")
        raw = s["kv"[which]][f][ids]
        if f == I4:
            low = (raw & 15).double()
            high = (raw >> 4).double()
            x = torch.empty(raw.shape[:-1] + (2 * raw.shape[-1],), dtype=torch.float64, device="cuda")
            x[..., 0::2], x[..., 1::2] = low - 16 * (low > 7), high - 16 * (high > 7)
        else:
            x = raw.view({F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8, FP8: torch.float8_e4m3fn}[f])
            x = x.to(torch.float32).double()
        if f in QMAX:
            x = x * s["scales"][f][ids, :, which].double()[:, :, None, None]
        parts.append(x.transpose(1, 2).reshape(-1, s["hkv"], s["d"]))
        at = end
    x = torch.cat(parts)
    return x[lo - pages[0] * P:hi - pages[0] * P]


def _code64(x, scale, fmt):
    """The format's value nearest to x over a 32-bit scale; the quotient is rounded to 32 bits first, as the
    format's definition says, and so decides the ties."""
    f = (x / scale).float().double() if scale > 0 else torch.zeros_like(x)
    if fmt == FP8:
        a = f.abs().clamp(max=448.0)
        unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
        return torch.sign(f) * torch.round(a / unit) * unit
    return torch.round(f).clamp(-QMAX[fmt], QMAX[fmt])


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rope":
        return _exact_rope(case, s)
    if op == "write" and s["fmt"] in QMAX:
        if len(s["seq_ids"]) * s["hkv"] / s["page"] + case["batch"] * s["hkv"] > 6000:
            return _exact_write_flat(case, s)
        return _exact_write(case, s)
    if op in ("write", "read"):
        if op == "write":  # unquantised pages hold the rounded rows
            seq, tok, dt = s["seq_ids"], s["token_ids"], torch.float32 if s["fmt"] == F32 else torch.bfloat16
            ids = torch.stack([s["table"][b, t // s["page"]] for b, t in zip(seq.tolist(), tok.tolist())]).long()
            for w in "kv":
                s[w][s["fmt"]].view(dt)[ids, :, tok % s["page"]] = s["new_" + w].to(dt)
        off, starts = s["back_off"].tolist(), s["back_starts"].tolist()
        k, v = (torch.cat([_stored64(s, b, starts[b], starts[b] + off[b + 1] - off[b], w) for b in range(len(starts))
                           if off[b + 1] > off[b]]) for w in (0, 1))
        return dict(k=k, v=v)
    return _exact_tree(case, s)


def _exact_rope(case, s):
    pos = s["rope_pos"].double()
    inv = s["inv_freq"]
    half = case["rot"] // 2
    c, n = torch.cos(torch.outer(pos, inv)).unsqueeze(1), torch.sin(torch.outer(pos, inv)).unsqueeze(1)

    def turn(x, w):
        y = x.double().clone()
        if w is not None:
            y *= w.double() / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / case["d"] + EPS)
        if case["pairs"] == "half":
            i, j = slice(0, half), slice(half, 2 * half)
        else:
            i, j = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
        z = y.clone()
        z[..., i] = y[..., i] * c - y[..., j] * n
        z[..., j] = y[..., i] * n + y[..., j] * c
        return z

    out = dict(q=turn(s["q"], s["qw"]))
    tok = s["token_ids"].long()
    ids = s["table"][s["seq_ids"].long(), tok // s["page"]].long()
    for name, rows in (("k", turn(s["new_k"], s["kw"])), ("v", s["new_v"].double())):
        pool = _stored(s, name).double()
        pool[ids, :, tok % s["page"], :] = rows
        out[name] = pool
    return out


def _exact_write(case, s):
    """Page by page and head by head."""
    fmt, P = s["fmt"], s["page"]
    off, starts, boff = s["off"].tolist(), s["starts"].tolist(), s["back_off"].tolist()
    scales = s["scales"][fmt].double().clone()
    out = dict(k=torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda"))
    out["v"] = out["k"].clone()
    for b in range(case["batch"]):
        a, n = starts[b], off[b + 1] - off[b]
        if n == 0:
            continue
        for which, name in ((0, "k"), (1, "v")):
            rows = s["new_" + name][off[b]:off[b + 1]].double()
            first = a - a % P
            held = _stored64(s, b, first, a, which) if a > first else rows[:0]
            for p in range(a // P, -(-(a + n) // P)):
                slot = int(s["table"][b, p])
                lo, hi = max(a, p * P), min(a + n, p * P + P)
                for g in range(s["hkv"]):
                    x = rows[lo - a:hi - a, g]
                    scale = float((x.abs().max() / QMAX[fmt]).float())
                    old = held[:, g] if lo > p * P else held[:0, g]
                    if len(old):
                        was = float(scales[slot, g, which])
                        if scale <= was:
                            scale = was
                        else:
                            old = _code64((old).float().double(), scale, fmt) * scale
                    y = torch.cat((old, _code64(x, scale, fmt) * scale))
                    scales[slot, g, which] = scale
                    i = boff[b] + p * P - first
                    out[name][i:i + len(y), g] = y
    out["scales"] = scales
    return out


def _exact_write_flat(case, s):
    """The same for many pages: the rows of all touched pages in one padded tensor."""
    fmt, P = s["fmt"], s["page"]
    off, starts, boff = s["off"].tolist(), s["starts"].tolist(), s["back_off"].tolist()
    scales = s["scales"][fmt].double().clone()
    out = {}
    for which, name in ((0, "k"), (1, "v")):
        y = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            a, n = starts[b], off[b + 1] - off[b]
            if n == 0:
                continue
            first = a - a % P
            pages = -(-(a + n - first) // P)
            ids = s["table"][b, first // P:first // P + pages].long()
            x = torch.zeros((pages * P, s["hkv"], s["d"]), dtype=torch.float64, device="cuda")
            x[a - first:a - first + n] = s["new_" + name][off[b]:off[b + 1]].double()
            x = x.view(pages, P, s["hkv"], s["d"])
            new = (x.abs().amax((1, 3)) / QMAX[fmt]).float().double()
            if a > first:
                was = scales[ids[0], :, which]
                held = _stored64(s, b, first, a, which)
                grown = torch.maximum(new[0], was)
                for g in range(s["hkv"]):
                    if grown[g] > was[g]:
                        held[:, g] = _code64(held[:, g].float().double(), float(grown[g]), fmt) * grown[g]
                new[0] = grown
            sc = new[:, None, :, None]
            f = torch.where(sc > 0, x / sc, 0 * x).float().double()
            if fmt == FP8:
                m = f.abs().clamp(max=448.0)
                unit = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
                f = torch.sign(f) * torch.round(m / unit) * unit
            else:
                f = torch.round(f).clamp(-QMAX[fmt], QMAX[fmt])
            z = (f * sc).reshape(pages * P, s["hkv"], s["d"])
            if a > first:
                z[:a - first] = held
            y[boff[b]:boff[b + 1]] = z[:a + n - first]
            scales[ids, :, which] = new
        out[name] = y
    out["scales"] = scales
    return out


def _exact_tree(case, s):
    batch, nq, hq, d = s["q"].shape
    group = hq // s["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    bits = 2 ** torch.arange(63, dtype=torch.int64, device="cuda")
    for b in range(batch):
        n, c = int(s["lens"][b]), int(s["drafts"][b])
        if c == 0:
            continue
        sees = torch.ones((c, n), dtype=torch.bool, device="cuda")
        m = s["mask"][b, :c, None]
        tree = torch.cat(((m & bits) != 0, m < 0), 1)[:, :c]
        sees[:, n - c:] = tree
        place = torch.arange(n, device="cuda")
        place[n - c:] = n - c + s["depth"][b, :c]
        K, V = _stored64(s, b, 0, n, 0), _stored64(s, b, 0, n, 1)
        for g in range(s["hkv"]):
            q = s["q"][b, :c, g * group:(g + 1) * group].double()
            x = torch.einsum("chd,nd->chn", q, K[:, g]) * d ** -0.5
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                far = (n - c + s["depth"][b, :c, None] - place[None]).double()
                x = x - s["slopes"][g * group:(g + 1) * group].double()[None, :, None] * far[:, None]
            x = torch.where(sees[:, None], x, torch.full_like(x, -math.inf))
            lse[b, :c, g * group:(g + 1) * group] = torch.logsumexp(x, -1)
            out[b, :c, g * group:(g + 1) * group] = torch.einsum("chn,nd->chd", torch.softmax(x, -1), V[:, g])
    return dict(out=out, lse=lse)
